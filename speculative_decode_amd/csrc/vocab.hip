// Operators over rows of vocabulary logits: log probabilities of given tokens with the
// entropy and the top alternatives of each row, and the distillation loss against a
// teacher's top alternatives with its gradient.
//
// A row z[0..V) with temperature T stands for q_i = e^{z_i/T} / sum_j e^{z_j/T}.  Everything
// is formed from the row's maximum m and sums of e_i = e^{(z_i - m)/T}:
//   log q_i = (z_i - m)/T - log S,                  S = sum e_i
//   entropy = log S + (sum e_i (m - z_i)/T) / S     (a sum of terms >= 0: nothing cancels)
// Sums are fp32 over a thread's terms (at most 136) and a tree over the workgroup's threads; what a
// row's slices or waves leave is added up in fp32 for the log probabilities (at most 33 slices)
// and in fp64 for the loss.
//
// What bounds them: each logit has to be read once (2 or 4 bytes) and costs one exponential
// and about ten vector operations, which at 2 bytes is close to the time of the read, so
// the two have to overlap.  A row is cut into slices of at most 4096 16-byte vectors; a
// workgroup of 256 threads holds a slice in registers (16 vectors a thread), so that the
// maximum, the sums and the selection all work on one read, and four workgroups share a
// compute unit: one loads while another computes.  A second small launch joins the slices.
//
// Vectors sit on 16-byte boundaries whatever the row's own alignment: vector v of a row
// holds elements v*EPV - off .. + EPV, where off counts the elements between the boundary
// at or below the row's start and that start.  Only a row's first and last vector can be
// partial; those are read element by element, with -inf in the places outside the row.
#include <math.h>

#include <type_traits>

#include "ssm_internal.h"

namespace mil {
namespace {

// Waits for LDS alone; loads and stores of global memory stay in flight across it
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

constexpr int kNT = 256;                  // threads of a slice workgroup
constexpr int kMaxVPT = 16;               // vectors per thread
constexpr int kSliceVecs = kNT * kMaxVPT; // vectors per slice
constexpr int kGroups = 128;              // groups (lane pairs) whose maxima bound the top-k threshold
constexpr int kHits = 512;                // vectors with candidates that a slice keeps in LDS
constexpr int kCand = 1024;               // and candidates
constexpr float kLog2e = 1.44269504088896340736f;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));  // 16 bytes that arrays keep in registers

template <bool BF>
struct Vec {
    static constexpr int EPV = BF ? 8 : 4;
    static constexpr int ELT = BF ? 2 : 4;
    __device__ static void unpack(u32x4 w, float (&f)[EPV]) {
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
        }
    }
    // round to the stored type (nearest even)
    __device__ static u32x4 pack(const float (&f)[EPV]) {
        u32x4 w;
        if constexpr (BF) {
            typedef __bf16 b2 __attribute__((ext_vector_type(2)));
            typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2){f[2 * i], f[2 * i + 1]}, b2));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
        }
        return w;
    }
};

// A row's vectors.  `base` is the 16-byte boundary at or below the row's first element.
struct Row {
    const char *row;
    int off, V, nv;
};
template <bool BF>
__device__ __forceinline__ Row open_row(const void *p, int64_t row, int64_t stride, int V) {
    Row r;
    r.row = static_cast<const char *>(p) + row * stride * Vec<BF>::ELT;
    r.off = (int)((reinterpret_cast<uintptr_t>(r.row) & 15) / Vec<BF>::ELT);
    r.V = V;
    r.nv = (r.off + V + Vec<BF>::EPV - 1) / Vec<BF>::EPV;
    return r;
}
template <bool BF>
__device__ __forceinline__ float row_elt(const Row &r, int e) {
    if constexpr (BF)
        return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(r.row)[e] << 16);
    else
        return reinterpret_cast<const float *>(r.row)[e];
}
template <bool BF>
__device__ __forceinline__ u32x4 load_vec(const Row &r, int v) {
    constexpr int EPV = Vec<BF>::EPV;
    const int e0 = v * EPV - r.off;
    if (e0 >= 0 && e0 + EPV <= r.V) {
        return *reinterpret_cast<const u32x4 *>(r.row + (int64_t)e0 * Vec<BF>::ELT);
    }
    float f[EPV];
#pragma unroll
    for (int i = 0; i < EPV; ++i) {
        const int e = e0 + i;
        f[i] = (e >= 0 && e < r.V) ? row_elt<BF>(r, e) : -INFINITY;
    }
    return Vec<BF>::pack(f);  // exact: the values are of the stored type
}
template <bool BF>
__device__ __forceinline__ u32x4 no_vec() {
    const uint32_t w = BF ? 0xff80ff80u : 0xff800000u;  // -inf everywhere
    return (u32x4){w, w, w, w};
}

// The vectors as they are again: without this the compiler keeps the values unpacked by one
// pass for the next, twice the registers, and half the workgroups fit a compute unit.
template <int VPT>
__device__ __forceinline__ void again(u32x4 (&raw)[VPT]) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) asm volatile("" : "+v"(raw[j]));
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Order of the alternatives: larger value first, -0 equal to +0, every NaN above every
// number, the lower id first among equals.  key32 is never 0, so 0 stands for "none".
__device__ __forceinline__ uint32_t key32(float f) {
    if (f != f) return 0xffffffffu;
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    if (k == 0xffffffffu) return __uint_as_float(0x7fc00000u);
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
__device__ __forceinline__ uint64_t full_key(float f, int id) {
    return ((uint64_t)key32(f) << 32) | (uint32_t)~id;
}

// Rank a list of distinct keys: `emit(rank, key)` for the k largest.  Two neighbouring lanes
// count for a key, each over every second other one.
template <typename F>
__device__ __forceinline__ void rank_list(const uint64_t *list, int n, int k, F emit) {
    for (int i = threadIdx.x >> 1; i < n; i += blockDim.x >> 1) {
        const uint64_t mine = list[i];
        int r = 0;
#pragma unroll 4
        for (int q = threadIdx.x & 1; q < n; q += 2) r += list[q] > mine;
        r += __shfl_xor(r, 1);
        if ((threadIdx.x & 1) == 0 && r < k) emit(r, mine);
    }
}

struct LogprobParams {
    const void *logits;
    int64_t stride;
    int rows, V, k, S, vps;  // slices per row, vectors per slice
    float T;
    const int32_t *tokens;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_lp;
    float4 *part;    // [rows][S]: maximum, S, sum of e (m - z) in log2 units
    uint64_t *keys;  // [rows][S][k] in falling order, 0 behind the last
};

// One slice: statistics and its own k best.
//
// Selection: the k-th largest of 128 group maxima is a lower bound of the slice's k-th
// largest value, and few elements are above it, so a look at each vector's maximum finds the
// vectors that hold candidates and a rank count orders those; no sort, and the result does
// not depend on the order in which candidates are collected since keys are distinct.  (With
// only what is above the bound as candidates, bf16 rows came up short at every second slice,
// their values being few: 512 rows of 128256, 20 alternatives, 63 us instead of 45.)  Where
// too many elements reach the bound (values clustered in few groups, or equal), or the slice
// holds a NaN, the exact k-th key is found by bisection over its 32 bits first, and elements
// equal to it are taken in rising id order as far as they are needed; so are masked ones.
//
// 4096 rows of 128256 bf16 values, 64 alternatives: 276 us with the joining launch, 1.05 GB at
// 3.8 TB/s, vector ALU 94 % busy.  128 rows, 20 alternatives: 20 us (1.7 TB/s), one round of
// workgroups: the chain of load, maximum, sums and selection.  One row: 13 us.
template <bool BF, int VPT>
__global__ __launch_bounds__(kNT, 4) void logprob_slice(const LogprobParams p) {
    constexpr int EPV = Vec<BF>::EPV;
    __shared__ float sMax[4], sLow[4];
    __shared__ __align__(16) float sG[kGroups];
    __shared__ float sSum[4][2];
    __shared__ uint64_t sCand[kCand];
    __shared__ int sCount, sHits, sBis[4];
    __shared__ u32x4 sHit[kHits];
    __shared__ int sHitAt[kHits];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t item = blockIdx.x;
    const int64_t row = item / p.S;
    const int s = (int)(item - row * p.S);
    const Row r = open_row<BF>(p.logits, row, p.stride, p.V);
    const int v0 = s * p.vps, v1 = min(v0 + p.vps, r.nv);

    u32x4 raw[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = v0 + j * kNT + tid;
        raw[j] = v < v1 ? load_vec<BF>(r, v) : no_vec<BF>();
    }
    if (tid == 0) sCount = 0, sHits = 0;
    float vm[VPT], tm = -INFINITY;  // each vector's maximum: the selection's only look at most of them
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float f[EPV];
        Vec<BF>::unpack(raw[j], f);
        vm[j] = f[0];
#pragma unroll
        for (int i = 1; i < EPV; ++i) vm[j] = fmaxf(vm[j], f[i]);
        tm = fmaxf(tm, vm[j]);
    }
    float gm = fmaxf(tm, __shfl_xor(tm, 1));
    if ((lane & 1) == 0) sG[wave * 32 + (lane >> 1)] = gm;
#pragma unroll
    for (int d = 2; d < 64; d <<= 1) gm = fmaxf(gm, __shfl_xor(gm, d));
    if (lane == 0) sMax[wave] = gm;
    __syncthreads();
    const float m = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
    const float mm = m == -INFINITY ? 0.f : m;
    const float c = kLog2e / p.T;
    float S = 0.f, W = 0.f;
    again(raw);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float f[EPV];
        Vec<BF>::unpack(raw[j], f);
#pragma unroll
        for (int i = 0; i < EPV; ++i) {
            // (e is 0 from far above -1000 on, and so is e d; the maximum keeps a NaN)
            const float d = __builtin_elementwise_maximum((f[i] - mm) * c, -1000.f);
            const float e = __builtin_amdgcn_exp2f(d);
            S += e;
            W = fmaf(e, -d, W);
        }
    }
    S = wave_sum(S);
    W = wave_sum(W);
    if (lane == 0) sSum[wave][0] = S, sSum[wave][1] = W;
    __syncthreads();
    S = (sSum[0][0] + sSum[1][0]) + (sSum[2][0] + sSum[3][0]);
    W = (sSum[0][1] + sSum[1][1]) + (sSum[2][1] + sSum[3][1]);
    if (tid == 0) p.part[item] = make_float4(m, S, W, 0.f);
    if (p.k == 0) return;

    // k-th largest group maximum: the smallest that fewer than k are above.  Two neighbouring
    // lanes count for a group, each over half the others.
    const int k = p.k;
    {
        const float g = sG[tid >> 1];
        const float *half = sG + (tid & 1) * (kGroups / 2);
        int more = 0;
#pragma unroll
        for (int q = 0; q < kGroups / 2; q += 4) {
            const float4 o = *reinterpret_cast<const float4 *>(half + q);
            more += (o.x > g) + (o.y > g) + (o.z > g) + (o.w > g);
        }
        more += __shfl_xor(more, 1);
        float low = more < k ? g : INFINITY;
#pragma unroll
        for (int d = 2; d < 64; d <<= 1) low = fminf(low, __shfl_xor(low, d));
        if (lane == 0) sLow[wave] = low;
    }
    __syncthreads();
    const float thr = fminf(fminf(sLow[0], sLow[1]), fminf(sLow[2], sLow[3]));
    const float least = fmaxf(thr, -3.402823466e38f);  // (masked elements are not candidates)
    bool exact = !(S == S);  // a NaN (or +inf) among the values
    if (!exact) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (vm[j] >= least) {  // above -inf, so inside the row
                const int at = atomicAdd(&sHits, 1);
                if (at < kHits) sHit[at] = raw[j], sHitAt[at] = (v0 + j * kNT + tid) * EPV - r.off;
            }
        }
        __syncthreads();
        // the few vectors with such elements, spread over all threads
        const int hits = sHits;
        exact = hits > kHits;
        if (!exact) {
            for (int x = tid; x < hits * EPV; x += kNT) {
                const int h = x / EPV, i = x % EPV;
                float f;
                if constexpr (BF)
                    f = __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(sHit + h)[i] << 16);
                else
                    f = reinterpret_cast<const float *>(sHit + h)[i];
                if (f >= least) {
                    const int at = atomicAdd(&sCount, 1);
                    if (at < kCand) sCand[at] = full_key(f, sHitAt[h] + i);
                }
            }
            __syncthreads();
            exact = sCount > kCand;
        }
    }
    // What is rarely needed reads the slice again, vector by vector, instead of keeping
    // registers for it: f(value, element) for every element of vector j of this thread that is
    // inside the row and the slice
    const int rounds = (v1 - v0 + kNT - 1) / kNT;
    auto each = [&](int j, auto f) {
        const int v = v0 + j * kNT + tid;
        if (v >= v1) return;
        float x[EPV];
        Vec<BF>::unpack(load_vec<BF>(r, v), x);
        const int e0 = v * EPV - r.off;
#pragma unroll
        for (int i = 0; i < EPV; ++i)
            if (e0 + i >= 0 && e0 + i < r.V) f(x[i], e0 + i);
    };
    uint32_t tkey = key32(thr);
    if (exact) {
        // the largest key that at least k elements reach (0: the slice has fewer than k)
        tkey = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t trial = tkey | (1u << bit);
            int n = 0;
            for (int j = 0; j < rounds; ++j) each(j, [&](float x, int) { n += key32(x) >= trial; });
#pragma unroll
            for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d);
            __syncthreads();
            if (lane == 0) sBis[wave] = n;
            __syncthreads();
            if (sBis[0] + sBis[1] + sBis[2] + sBis[3] >= k) tkey = trial;
        }
        __syncthreads();
        if (tid == 0) sCount = 0;
        __syncthreads();
        for (int j = 0; j < rounds; ++j)
            each(j, [&](float x, int e) {
                if (key32(x) > tkey) {  // fewer than k of them
                    const int at = atomicAdd(&sCount, 1);
                    if (at < kCand) sCand[at] = full_key(x, e);
                }
            });
        __syncthreads();
    }
    int n = sCount;
    if (n < k && tkey != 0) {
        // the k-th value is the bound itself: its elements in rising id order, as many as
        // are missing.  Vector j of all threads comes before vector j + 1 of any.
        const int want = k - n;
        int got = 0;
        for (int j = 0; j < rounds && got < want; ++j) {
            int mine = 0;
            each(j, [&](float x, int) { mine += key32(x) == tkey; });
            int upto = mine;  // inclusive count over lanes
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d);
                if (lane >= d) upto += o;
            }
            __syncthreads();
            if (lane == 63) sBis[wave] = upto;
            __syncthreads();
            int at = got + upto - mine;
            for (int w = 0; w < wave; ++w) at += sBis[w];
            got += sBis[0] + sBis[1] + sBis[2] + sBis[3];
            if (mine)
                each(j, [&](float x, int e) {
                    if (key32(x) == tkey) {
                        if (at < want) sCand[n + at] = full_key(x, e);  // n + at < k <= 64
                        ++at;
                    }
                });
        }
        n += min(got, want);
        __syncthreads();
    }
    uint64_t *keys = p.keys + item * k;
    for (int i = tid; i < k; i += kNT)
        if (i >= n) keys[i] = 0;
    rank_list(sCand, n, k, [&](int rank, uint64_t key) { keys[rank] = key; });
}

// Join a row's slices: one workgroup per row.  6 us for 128 rows, 15 for 4096 with 64 alternatives.
template <bool BF>
__global__ __launch_bounds__(kNT) void logprob_join(const LogprobParams p) {
    extern __shared__ uint64_t sKeys[];  // [S * k] and as many again
    __shared__ int sCount;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, k = p.k, SK = p.S * p.k;
    float m = -INFINITY;
    for (int s = 0; s < p.S; ++s) m = fmaxf(m, p.part[row * p.S + s].x);
    const float c = kLog2e / p.T;
    float S = 0.f, W = 0.f;
    for (int s = 0; s < p.S; ++s) {
        const float4 q = p.part[row * p.S + s];
        if (q.x == -INFINITY && q.y == 0.f) continue;  // nothing in this slice
        // bounded: a slice of masks of the lowest value is an infinite number of steps below
        const float up = fminf((m - q.x) * c, 1e30f), f = __builtin_amdgcn_exp2f(-up);
        S += f * q.y;
        W += f * fmaf(up, q.y, q.z);
    }
    const bool empty = m == -INFINITY && S == 0.f;
    const float logS = logf(S);
    if (tid == 0) {
        if (p.entropy) p.entropy[row] = empty ? 0.f : logS + (W / S) * 0.69314718055994530942f;
        if (p.logprob) {
            const int tok = p.tokens[row];
            float lp = 0.f;
            if (tok >= p.V)
                lp = __uint_as_float(0x7fc00000u);
            else if (tok >= 0) {
                const Row r = open_row<BF>(p.logits, row, p.stride, p.V);
                lp = empty ? -INFINITY : (row_elt<BF>(r, tok) - m) / p.T - logS;
            }
            p.logprob[row] = lp;
        }
    }
    if (k == 0) return;
    auto emit = [&](int rank, uint64_t key) {
        const float z = key_value((uint32_t)(key >> 32));
        p.top_ids[row * k + rank] = (int32_t)~(uint32_t)key;
        p.top_lp[row * k + rank] = empty ? -INFINITY : (z - m) / p.T - logS;
    };
    const uint64_t *keys = p.keys + row * SK;
    if (p.S == 1) {
        for (int i = tid; i < k; i += kNT) emit(i, keys[i]);
        return;
    }
    // each slice's list is in falling order: its element d - 1 with S * d >= k bounds the
    // row's k-th key from below
    const int d = (k + p.S - 1) / p.S;
    uint64_t *sList = sKeys + SK;
    for (int i = tid; i < SK; i += kNT) sKeys[i] = keys[i];
    if (tid == 0) sCount = 0;
    __syncthreads();
    uint64_t thr = ~0ull;
    for (int s = 0; s < p.S; ++s) thr = min(thr, sKeys[s * k + d - 1]);
    for (int i = tid; i < SK; i += kNT)
        if (sKeys[i] >= thr && sKeys[i] != 0) sList[atomicAdd(&sCount, 1)] = sKeys[i];
    __syncthreads();
    rank_list(sList, sCount, k, emit);
}

// ------------------------------------------------------------------- distillation
//
// p: the teacher's probabilities at the row's k alternatives (a double id's are added up),
// q: the student's.  With the tail, everything else is one more outcome with p_t = 1 - sum p
// and q_t = sum of q outside the alternatives; without, p is divided by its sum.
//   loss       = sum p log(p/q) (+ p_t log(p_t/q_t))
//   dloss/dz_i = (q_i - p_i)/T at the alternatives,  (q_i - p_t q_i/q_t)/T (or q_i/T) elsewhere
// What lies outside the alternatives is summed directly, never as 1 - sum q, and relative to its
// own greatest logit m_r: with r_i = e^{(z_i - m_r)/T} and R = sum r_i there,
//   log q_t = (m_r - m)/T + log R - log Z,    gradient there = r_i ((q_t - p_t)/R)/T
// hold however far it lies below the alternatives (relative to the row's maximum it is 0 in fp32
// from 87 T down): no factor is above 1, and -inf gives 0.
// The alternatives are few: lane q of every wave knows where alternative q lies (which vector,
// of which wave and lane), and a wave that comes to a vector asks by one ballot whether there
// are any in its 64; one in four has.  They are taken out of the vectors (-inf in their place)
// before anything is summed.
struct DistillParams {
    const void *logits;
    int64_t stride;
    int rows, V, k, S, vps, tail;
    float T;
    const int32_t *ids;
    const float *lp;
    float *loss;
    float4 *part;   // [rows][S]: outside the alternatives, the maximum and the sum relative to it
    float4 *stats;  // [rows]: maximum outside, (q_t - p_t)/R, the row's maximum, 1/Z (-1: no alternatives)
    const float *grad;
    void *out;
    int64_t out_stride;
};

// The teacher's side of a row, in one wave: lane j < k holds alternative j.  p is 0 for
// absent ones and for all but the first of a repeated id.
struct Teacher {
    int id;
    double p, total;
    bool any, bad;  // some alternative present; an id behind the vocabulary or a NaN
};
__device__ __forceinline__ Teacher teacher(const DistillParams &a, int64_t row, int lane) {
    Teacher t;
    t.id = lane < a.k ? a.ids[row * a.k + lane] : -1;
    t.bad = __ballot(t.id >= a.V) != 0;
    if (t.id >= a.V) t.id = -1;
    const double mine = t.id >= 0 ? exp((double)a.lp[row * a.k + lane]) : 0.0;
    t.bad |= __ballot(mine != mine) != 0;
    double sum = 0.0;
    bool later = false;
    for (int q = 0; q < a.k; ++q) {
        const int o = __shfl(t.id, q);
        const double v = __shfl(mine, q);
        if (o == t.id) {
            sum += v;
            later |= q < lane;
        }
    }
    t.p = (t.id < 0 || later) ? 0.0 : sum;
    t.total = wave_sum(t.p);
    t.any = __ballot(t.id >= 0) != 0 && t.total > 0.0;
    if (!a.tail && t.any) t.p /= t.total;
    if (later) t.id = -1;  // the first of a repeated id stands for all
    return t;
}
// What a row's loss and gradient are made of
struct RowEnd {
    float loss, m, slope;  // slope: of the gradient outside the alternatives, (q_t - p_t)/R
    double Z;              // sum of e^{(z-m)/T} over the whole row (0: all of it is masked)
};
// From the greatest logit outside the alternatives, R = sum of e^{(z-m_r)/T} there, and each lane's
// own alternative's logit.  A NaN or +inf anywhere makes Z a NaN, and with it everything.
__device__ __forceinline__ RowEnd row_end(const DistillParams &a, const Teacher &t, float zj, float mr, double R) {
    RowEnd o;
    o.m = fmaxf(mr, wave_max(t.id >= 0 ? zj : -INFINITY));
    if (o.m == -INFINITY) o.m = 0.f;
    const double T = (double)a.T, dj = ((double)zj - (double)o.m) / T, below = ((double)mr - (double)o.m) / T;
    const double rest = R == 0.0 ? 0.0 : R * exp(below);
    // (fp32 will do: an argument's rounding, 2^-24 |d| of e^d, is largest at d = -1)
    o.Z = (double)wave_sum(t.id >= 0 ? expf((float)dj) : 0.f) + rest;
    const double pt = a.tail ? fmax(0.0, 1.0 - t.total) : 0.0;
    o.slope = (float)(R == 0.0 ? 0.0 * o.Z : (rest / o.Z - pt) / R);
    // p log(p/q) = p (log(p Z) - (z-m)/T), and so for the tail
    double l = t.p > 0.0 ? (o.Z == 0.0 ? (double)INFINITY : t.p * (log(t.p * o.Z) - dj)) : 0.0;
    l = wave_sum(l);
    if (pt > 0.0 && R > 0.0) l += pt * (log(pt * o.Z / R) - below);
    o.loss = (float)l;
    return o;
}

// Where this lane's alternative lies among the vectors of a workgroup with STEP threads (vector
// j * STEP + thread): round j (-1: not with this wave), lane, and place in the vector
struct Spot {
    int j, lane, i;
};
template <int EPV, int STEP>
__device__ __forceinline__ Spot spot_of(int id, int off, int v0, int v1, int wave) {
    const int at = id + off, v = at / EPV - v0;
    Spot s;
    const bool mine = id >= 0 && v >= 0 && v < v1 - v0 && (v % STEP) / 64 == wave;
    s.j = mine ? v / STEP : -1;
    s.lane = v % 64;
    s.i = at % EPV;
    return s;
}
// f(number of the alternative, its place in the vector, whether it is this lane's) for each of the
// alternatives in vector j of this wave's lanes.  Number and place are uniform.
template <typename F>
__device__ __forceinline__ void at_spots(const Spot &s, int j, F f) {
    // one vector after another: with several under way at once the registers run out
    __builtin_amdgcn_sched_barrier(0);
    int own = s.j;
    asm volatile("" : "+v"(own));
    for (uint64_t some = __ballot(own == j); some; some &= some - 1) {
        const int q = __builtin_ctzll(some);
        f(q, __builtin_amdgcn_readlane(s.i, q), __builtin_amdgcn_readlane(s.lane, q) == (int)(threadIdx.x & 63));
    }
}
// (z - m) * log2(e)/T with the constant in two parts: its rounding alone would move every
// exponential of the row the same way, which the loss, a small difference of large terms,
// shows.  Both parts are positive, so that z = -inf gives -inf and a NaN stays one.
struct Scale {
    float hi, lo;
};
__device__ __forceinline__ Scale scale_of(float T) {
    const double c = 1.4426950408889634074 / (double)T;
    Scale s;
    s.hi = (float)c;
    if ((double)s.hi >= c) s.hi = __uint_as_float(__float_as_uint(s.hi) - 1);
    s.lo = (float)(c - (double)s.hi);
    return s;
}
__device__ __forceinline__ float exp_of(float z, float m, const Scale &c) {
    const float d = z - m;
    return __builtin_amdgcn_exp2f(fmaf(d, c.lo, d * c.hi));
}

// -inf in the place of the alternatives in vector j
template <bool BF>
__device__ __forceinline__ void take_out(u32x4 &raw, const Spot &spot, int j) {
    constexpr int EPV = Vec<BF>::EPV;
    at_spots(spot, j, [&](int, int place, bool mine) {
#pragma unroll
        for (int i = 0; i < EPV; ++i)
            if (place == i) {
                constexpr int per = BF ? 2 : 1;
                const uint32_t w = raw[i / per];
                const uint32_t out = !BF ? 0xff800000u
                                     : i % per ? (w & 0xffffu) | 0xff800000u
                                               : (w & 0xffff0000u) | 0xff80u;
                raw[i / per] = mine ? out : w;
            }
    });
}
// Sum of one vector
template <bool BF>
__device__ __forceinline__ float sum_vec(u32x4 raw, float m, const Scale &c) {
    constexpr int EPV = Vec<BF>::EPV;
    float f[EPV];
    Vec<BF>::unpack(raw, f);
#pragma unroll
    for (int i = 0; i < EPV; ++i) f[i] = exp_of(f[i], m, c);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < EPV; ++i) sum += f[i];
    asm volatile("" : "+v"(sum));  // now: put off to where the sum is used, the terms of all vectors would wait
    __builtin_amdgcn_sched_barrier(0);  // and one vector after another, for the same reason
    return sum;
}

// Sums of a slice.  515 rows of 32003 fp32 values: 24 us (67 MB at 2.8 TB/s), the gradient's launch
// below 23 (133 MB at 5.8 TB/s).
template <bool BF, int VPT>
__global__ __launch_bounds__(kNT, 4) void distill_slice(const DistillParams p) {
    constexpr int EPV = Vec<BF>::EPV;
    __shared__ float sMax[4], sSum[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t item = blockIdx.x;
    const int64_t row = item / p.S;
    const int s = (int)(item - row * p.S);
    const Row r = open_row<BF>(p.logits, row, p.stride, p.V);
    const int v0 = s * p.vps, v1 = min(v0 + p.vps, r.nv);
    // (asked for first: the vectors are looked at as they arrive, which takes the alternatives)
    const int id = lane < p.k ? p.ids[row * p.k + lane] : -1;
    u32x4 raw[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = v0 + j * kNT + tid;
        raw[j] = v < v1 ? load_vec<BF>(r, v) : no_vec<BF>();
    }
    const Spot spot = spot_of<EPV, kNT>(id < p.V ? id : -1, r.off, v0, v1, wave);
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPT; ++j) take_out<BF>(raw[j], spot, j);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        float f[EPV];
        Vec<BF>::unpack(raw[j], f);
#pragma unroll
        for (int i = 0; i < EPV; ++i) m = fmaxf(m, f[i]);
    }
    m = wave_max(m);
    if (lane == 0) sMax[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sMax[0], sMax[1]), fmaxf(sMax[2], sMax[3]));
    const float mm = m == -INFINITY ? 0.f : m;
    const Scale c = scale_of(p.T);
    float rest = 0.f;
    again(raw);
#pragma unroll
    for (int j = 0; j < VPT; ++j) rest += sum_vec<BF>(raw[j], mm, c);
    rest = wave_sum(rest);
    if (lane == 0) sSum[wave] = rest;
    __syncthreads();
    if (tid == 0) p.part[item] = make_float4(m, (sSum[0] + sSum[1]) + (sSum[2] + sSum[3]), 0.f, 0.f);
}

// Loss of a row from its slices: one wave per row.  7 us for 515 rows.
template <bool BF>
__global__ __launch_bounds__(kNT) void distill_join(const DistillParams p) {
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * (kNT / 64) + (threadIdx.x >> 6);
    if (row >= p.rows) return;
    const Teacher t = teacher(p, row, lane);
    float m = -INFINITY;
    for (int s = 0; s < p.S; ++s) m = fmaxf(m, p.part[row * p.S + s].x);
    double R = 0.0;
    for (int s = 0; s < p.S; ++s) {
        const float4 q = p.part[row * p.S + s];
        if (q.x == -INFINITY && q.y == 0.f) continue;  // nothing in this slice
        R += exp(((double)q.x - (double)m) / (double)p.T) * (double)q.y;
    }
    const Row r = open_row<BF>(p.logits, row, p.stride, p.V);
    const RowEnd o = row_end(p, t, t.id >= 0 ? row_elt<BF>(r, t.id) : 0.f, m, R);
    if (lane == 0) {
        const float nan = __uint_as_float(0x7fc00000u);
        p.loss[row] = t.bad ? nan : t.any ? o.loss : 0.f;
        p.stats[row] = make_float4(m == -INFINITY ? 0.f : m, t.bad ? nan : o.slope, o.m,
                                   t.bad ? nan : !t.any ? -1.f : o.Z == 0.0 ? 0.f : (float)(1.0 / o.Z));
    }
}

// One vector of the gradient
template <bool BF>
__device__ __forceinline__ void store_vec(char *orow, int ooff, int off, int V, int e0, const float (&g)[Vec<BF>::EPV]) {
    constexpr int EPV = Vec<BF>::EPV;
    const u32x4 w = Vec<BF>::pack(g);
    if (ooff == off && e0 >= 0 && e0 + EPV <= V) {
        *reinterpret_cast<u32x4 *>(orow + (int64_t)e0 * Vec<BF>::ELT) = w;
        return;
    }
#pragma unroll
    for (int i = 0; i < EPV; ++i) {
        const int e = e0 + i;
        if (e < 0 || e >= V) continue;
        if constexpr (BF)
            reinterpret_cast<uint16_t *>(orow)[e] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
        else
            reinterpret_cast<uint32_t *>(orow)[e] = w[i];
    }
}
// Gradient of one vector of logits: wr e^{(z-m)c}, m the maximum outside the alternatives, and
// own(q, z) at alternative q.  (Here the constant in one part will do: it moves a probability by
// no more than its own argument's rounding.)
template <bool BF, typename F>
__device__ __forceinline__ void grad_vec(u32x4 raw, const Spot &spot, int j, float m, float c, float wr, F own,
                                         float (&g)[Vec<BF>::EPV]) {
    constexpr int EPV = Vec<BF>::EPV;
    float f[EPV];
    Vec<BF>::unpack(raw, f);
#pragma unroll
    for (int i = 0; i < EPV; ++i) g[i] = __builtin_amdgcn_exp2f((f[i] - m) * c) * wr;
    at_spots(spot, j, [&](int q, int place, bool mine) {
#pragma unroll
        for (int i = 0; i < EPV; ++i)
            if (place == i) {
                const float v = own(q, f[i]);
                g[i] = mine ? v : g[i];
            }
    });
}
// The value of one lane, the same for all
__device__ __forceinline__ float of_lane(float v, int q) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), q));
}

template <bool BF, int VPT>
__global__ __launch_bounds__(kNT, 4) void distill_grad(const DistillParams p) {
    constexpr int EPV = Vec<BF>::EPV;
    __shared__ int sId[64];
    __shared__ float sP[64];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t item = blockIdx.x;
    const int64_t row = item / p.S;
    const int s = (int)(item - row * p.S);
    const Row r = open_row<BF>(p.logits, row, p.stride, p.V);
    const int v0 = s * p.vps, v1 = min(v0 + p.vps, r.nv);
    u32x4 raw[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int v = v0 + j * kNT + tid;
        raw[j] = v < v1 ? load_vec<BF>(r, v) : no_vec<BF>();
    }
    if (wave == 0) {
        const Teacher t = teacher(p, row, lane);
        sId[lane] = t.id;
        sP[lane] = (float)t.p;
    }
    lds_barrier();
    const Spot spot = spot_of<EPV, kNT>(sId[lane], r.off, v0, v1, wave);
    const float pj = sP[lane];
    const float4 st = p.stats[row];
    const float c = kLog2e / p.T;
    const float w = p.grad[row] / p.T, wq = w * st.w, wr = w * st.y, wp = w * pj;
    char *orow = static_cast<char *>(p.out) + row * p.out_stride * Vec<BF>::ELT;
    const int ooff = (int)((reinterpret_cast<uintptr_t>(orow) & 15) / Vec<BF>::ELT);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int q = j * kNT + tid;
        float g[EPV];
        // (an alternative's logit as it was loaded: out may be the logits, and the workgroup of
        // another slice through with them)
        grad_vec<BF>(raw[j], spot, j, st.x, c, wr,
                     [&](int q, float z) { return __builtin_amdgcn_exp2f((z - st.z) * c) * wq - of_lane(wp, q); }, g);
        if (st.w < 0.f) {  // no alternatives: zeros, whatever the logits hold
#pragma unroll
            for (int i = 0; i < EPV; ++i) g[i] = 0.f;
        }
        if (v0 + q < v1) store_vec<BF>(orow, ooff, r.off, r.V, (v0 + q) * EPV - r.off, g);
    }
}

// Loss and gradient in one pass.  A workgroup holds a whole row in the registers of its waves
// but one (15 waves of 17 vectors a thread hold 130560 bf16 values in half of their 128
// registers) and walks over the rows.  While it stores the gradient of one row it asks for
// the next: a vector's registers are free once its gradient is formed.  The last wave holds no
// logits: it prepares the teacher's side of the next row and works out the loss of this one,
// in double precision, while the others are busy with the gradient.  Rows start and end on
// 16-byte boundaries.  4096 rows of 128256 bf16 values with 64 alternatives: 492 us, 2.12 GB at 4.3
// TB/s, 0.70 of the rate of an elementwise pass over as much (vector ALU 59 % busy): a row's
// maximum, sums and gradient follow one another, and only the gradient's part of them stores, and
// loads the next row.
struct RowTeacher {
    int id[64];
    float p[64], z[64];
    float top;  // the greatest z
    double total;
    int kind;  // 0: no alternatives, 1: some, 2: an id behind the vocabulary or a NaN
};
// waves per SIMD that the registers of a workgroup leave room for
constexpr int rows_waves(int vpt) { return vpt <= 5 ? 6 : 4; }
template <bool BF, int NW, int VPT>
__global__ __launch_bounds__(NW * 64, rows_waves(VPT)) void distill_rows(const DistillParams p) {
    constexpr int EPV = Vec<BF>::EPV, MW = NW - 1, NT = MW * 64;
    __shared__ RowTeacher sT[2];
    __shared__ float sMax[MW], sSum[MW];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nv = p.V / EPV;
    if (wave == MW) {
        Teacher t{};
        auto prepare = [&](int64_t row, int at) {
            t = teacher(p, row, lane);
            RowTeacher &o = sT[at];
            o.id[lane] = t.id;
            o.p[lane] = (float)t.p;
            const float z = t.id >= 0 ? row_elt<BF>(open_row<BF>(p.logits, row, p.stride, p.V), t.id) : -INFINITY;
            o.z[lane] = z;
            const float top = wave_max(z);
            if (lane == 0) o.top = top, o.total = t.total, o.kind = t.bad ? 2 : t.any;
        };
        prepare(blockIdx.x, 0);
        lds_barrier();
        int at = 0;
        for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, at ^= 1) {
            lds_barrier();
            lds_barrier();
            float m = -INFINITY;
            double R = 0.0;
            for (int i = 0; i < MW; ++i) m = fmaxf(m, sMax[i]), R += (double)sSum[i];
            const RowEnd o = row_end(p, t, sT[at].z[lane], m, R);
            if (lane == 0) p.loss[row] = t.bad ? __uint_as_float(0x7fc00000u) : t.any ? o.loss : 0.f;
            if (row + gridDim.x < p.rows) prepare(row + gridDim.x, at ^ 1);
            lds_barrier();
        }
        return;
    }
    const Scale c = scale_of(p.T);
    const float c1 = kLog2e / p.T;
    u32x4 raw[VPT];
    // a row as a bounded view: what lies behind it reads as zero (and is passed over), and is
    // not written; one offset per lane serves all vectors
    auto view = [&](const void *base, int64_t row, int64_t stride) {
        return __builtin_amdgcn_make_buffer_rsrc(
            const_cast<char *>(static_cast<const char *>(base)) + row * stride * Vec<BF>::ELT, (short)0, nv * 16,
            0x00020000);
    };
    auto ask = [&](int j, __amdgpu_buffer_rsrc_t r) {
        raw[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, tid * 16, j * NT * 16, 0));
    };
    int64_t row = blockIdx.x;
#pragma unroll
    for (int j = 0; j < VPT; ++j) ask(j, view(p.logits, row, p.stride));
    lds_barrier();
    for (int at = 0; row < p.rows; row += gridDim.x, at ^= 1) {
        const RowTeacher &t = sT[at];
        const Spot spot = spot_of<EPV, NT>(t.id[lane], 0, 0, nv, wave);
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPT; ++j) take_out<BF>(raw[j], spot, j);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (j * NT + tid >= nv) continue;
            float f[EPV];
            Vec<BF>::unpack(raw[j], f);
#pragma unroll
            for (int i = 0; i < EPV; ++i) m = fmaxf(m, f[i]);
        }
        m = wave_max(m);
        if (lane == 0) sMax[wave] = m;
        lds_barrier();
        for (int i = 0; i < MW; ++i) m = fmaxf(m, sMax[i]);
        const float whole = fmaxf(m, t.top), mw = whole == -INFINITY ? 0.f : whole;
        const float below = m == -INFINITY ? 0.f : exp_of(m, mw, c);
        m = m == -INFINITY ? 0.f : m;
        float rest = 0.f;
        again(raw);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const float sum = sum_vec<BF>(raw[j], m, c);
            rest += j * NT + tid < nv ? sum : 0.f;
        }
        rest = wave_sum(rest);
        if (lane == 0) sSum[wave] = rest;
        const float own = exp_of(t.z[lane], mw, c), top = wave_sum(own);  // (0 where there is no alternative)
        lds_barrier();
        double R = 0.0;
#pragma unroll 1
        for (int i = 0; i < MW; ++i) R += (double)sSum[i];
        // as in row_end (what `below` loses under 2^-126 is nothing beside what is added to it)
        const double rw = R * (double)below, Z = (double)top + rw;
        const int kind = t.kind;
        const double pt = p.tail ? fmax(0.0, 1.0 - t.total) : 0.0;
        const float w = kind == 2 ? __uint_as_float(0x7fc00000u) : p.grad[row] / p.T;
        const float wr = w * (float)(R == 0.0 ? 0.0 * Z : (rw / Z - pt) / R);
        const float gq = own * (Z == 0.0 ? 0.f : (float)((double)w / Z)) - w * t.p[lane];
        const int64_t next = row + gridDim.x;
        const __amdgpu_buffer_rsrc_t out = view(p.out, row, p.out_stride);
        const __amdgpu_buffer_rsrc_t in = view(p.logits, next < p.rows ? next : row, p.stride);
        again(raw);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float g[EPV];
            grad_vec<BF>(raw[j], spot, j, m, c1, wr, [&](int q, float) { return of_lane(gq, q); }, g);
            u32x4 o = Vec<BF>::pack(g);
            if (kind == 0) o = (u32x4){};
            __builtin_amdgcn_raw_buffer_store_b128(o, out, tid * 16, j * NT * 16, 0);
            if (next < p.rows) ask(j, in);
        }
        lds_barrier();
    }
}

// Slices per row and vectors per slice: as few slices as hold the row, more (down to 512
// vectors a slice) while the launch has fewer workgroups than four per compute unit, or than
// eight where half the registers a thread would let more of them in (log probabilities, 256
// rows of 128256: 4 slices 46 us, 8 slices 38; 128 rows: 4 slices 37, 8 slices 29, 16 slices 32).
void cut(int64_t rows, int V, bool bf, int *S, int *vps) {
    const int epv = bf ? 8 : 4;
    const int nv = (V + 2 * (epv - 1)) / epv;  // whatever the alignment
    int s = (nv + kSliceVecs - 1) / kSliceVecs;
    while (rows * s < ((nv + s - 1) / s > kSliceVecs / 2 ? 2048 : 1024) && s < 16 && (nv + 2 * s - 1) / (2 * s) >= 512)
        s *= 2;
    *S = s;
    *vps = (nv + s - 1) / s;
}

#define MIL_BY_SIZE(kernel)                                                                     \
    template <typename P>                                                                       \
    hipError_t run_##kernel(bool bf, int vps, unsigned grid, const P &p, hipStream_t s) {       \
        const int vpt = (vps + kNT - 1) / kNT;                                                  \
        auto go = [&](auto n) {                                                                 \
            constexpr int VPT = decltype(n)::value;                                             \
            if (bf)                                                                             \
                hipLaunchKernelGGL((kernel<true, VPT>), dim3(grid), dim3(kNT), 0, s, p);        \
            else                                                                                \
                hipLaunchKernelGGL((kernel<false, VPT>), dim3(grid), dim3(kNT), 0, s, p);       \
        };                                                                                      \
        if (vpt <= 2)                                                                           \
            go(std::integral_constant<int, 2>{});                                               \
        else if (vpt <= 4)                                                                      \
            go(std::integral_constant<int, 4>{});                                               \
        else if (vpt <= 8)                                                                      \
            go(std::integral_constant<int, 8>{});                                               \
        else                                                                                    \
            go(std::integral_constant<int, 16>{});                                              \
        return hipGetLastError();                                                               \
    }
MIL_BY_SIZE(logprob_slice)
MIL_BY_SIZE(distill_slice)
MIL_BY_SIZE(distill_grad)

// Rows that one workgroup holds whole (distill_rows): up to what fits, in vectors.  Against the
// three launches of the separate calls (loss with gradient, bf16, us): 4096 rows of 128256 492 :
// 635, of 32000 151 : 209, of 8192 54 : 75; 128 rows of 32000 15 : 21.  Short rows in large
// numbers wait for one another (4096 rows of 1000 60 : 48, 2048 rows 33 : 29, 1024 rows 22 : 23).
// A few rows of 128256 are the one place where the slices' more workgroups are ahead (4 rows
// 25 : 21), not far enough for a rule of its own.
constexpr int kWholeMin = 512, kWholeMax = 15 * 64 * 17, kWholeRows = 1024;
hipError_t run_distill_rows(bool bf, int nv, const DistillParams &p, hipStream_t s) {
    int dev = 0, cus = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e == hipSuccess) e = hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev);
    if (e != hipSuccess) return e;
    auto go = [&](auto nw, auto n) {
        constexpr int NW = decltype(nw)::value, VPT = decltype(n)::value;
        const int most = cus * rows_waves(VPT) * 4 / NW;
        const unsigned grid = (unsigned)(p.rows < most ? p.rows : most);
        if (bf)
            hipLaunchKernelGGL((distill_rows<true, NW, VPT>), dim3(grid), dim3(NW * 64), 0, s, p);
        else
            hipLaunchKernelGGL((distill_rows<false, NW, VPT>), dim3(grid), dim3(NW * 64), 0, s, p);
    };
    const std::integral_constant<int, 8> w8;
    const std::integral_constant<int, 16> w16;
    // Eight waves, and two or three workgroups on a compute unit, as far as they hold a row (16384
    // bf16 values, 4096 rows: 69 us, with one workgroup of 16 waves 182); the vectors a thread in
    // steps, since those without a value still cost their share of the work (32000 values, 64
    // alternatives: 9 vectors 151 us, as many in twice the waves 266)
    const int each = (nv + 7 * 64 - 1) / (7 * 64);
    if (each <= 3)
        go(w8, std::integral_constant<int, 3>{});
    else if (each <= 5)
        go(w8, std::integral_constant<int, 5>{});
    else if (each <= 9)
        go(w8, std::integral_constant<int, 9>{});
    else if (each <= 13)
        go(w8, std::integral_constant<int, 13>{});
    else if (each <= 17)
        go(w8, std::integral_constant<int, 17>{});
    else if (nv <= 15 * 64 * 9)
        go(w16, std::integral_constant<int, 9>{});
    else if (nv <= 15 * 64 * 13)
        go(w16, std::integral_constant<int, 13>{});
    else
        go(w16, std::integral_constant<int, 17>{});
    return hipGetLastError();
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }

}  // namespace

bool vocab_supported(int64_t rows, int V, bool bf) {
    // (at most bytes / 64 KiB + 2 slices of kNT threads a row, or 2048 workgroups where there are
    // few rows: under 2^32 threads)
    return V <= MIL_VOCAB_MAX && rows * (2 + ((int64_t)V * (bf ? 2 : 4) >> 16)) < 1 << 24;
}

int64_t logprobs_workspace_bytes(int rows, int V, bool bf, int k) {
    int S, vps;
    cut(rows, V, bf, &S, &vps);
    return up256((int64_t)rows * S * sizeof(float4)) + up256((int64_t)rows * S * k * 8);
}

hipError_t launch_logprobs(const void *logits, int rows, int V, int64_t stride, bool bf, float T,
                           const int32_t *tokens, int k, float *logprob, float *entropy, int32_t *top_ids,
                           float *top_lp, void *ws, hipStream_t s) {
    LogprobParams p{};
    p.logits = logits, p.stride = stride, p.rows = rows, p.V = V, p.k = k, p.T = T;
    p.tokens = tokens, p.logprob = logprob, p.entropy = entropy, p.top_ids = top_ids, p.top_lp = top_lp;
    cut(rows, V, bf, &p.S, &p.vps);
    p.part = static_cast<float4 *>(ws);
    p.keys = reinterpret_cast<uint64_t *>(static_cast<char *>(ws) + up256((int64_t)rows * p.S * sizeof(float4)));
    hipError_t e = run_logprob_slice(bf, p.vps, (unsigned)((int64_t)rows * p.S), p, s);
    if (e != hipSuccess) return e;
    const size_t lds = (p.S > 1 ? 2 : 0) * (size_t)p.S * k * 8;
    if (bf)
        hipLaunchKernelGGL(logprob_join<true>, dim3(rows), dim3(kNT), lds, s, p);
    else
        hipLaunchKernelGGL(logprob_join<false>, dim3(rows), dim3(kNT), lds, s, p);
    return hipGetLastError();
}

int64_t distill_workspace_bytes(int rows, int V, bool bf) {
    int S, vps;
    cut(rows, V, bf, &S, &vps);
    return up256((int64_t)rows * S * sizeof(float4)) + up256((int64_t)rows * sizeof(float4));
}

namespace {
DistillParams distill_params(const void *logits, int rows, int V, int64_t stride, bool bf, float T, const int32_t *ids,
                             const float *lp, int k, bool tail) {
    DistillParams p{};
    p.logits = logits, p.stride = stride, p.rows = rows, p.V = V, p.k = k, p.tail = tail, p.T = T;
    p.ids = ids, p.lp = lp;
    cut(rows, V, bf, &p.S, &p.vps);
    return p;
}
}  // namespace

hipError_t launch_distill_forward(const void *logits, int rows, int V, int64_t stride, bool bf, float T,
                                  const int32_t *ids, const float *lp, int k, bool tail, float *loss, float *stats,
                                  void *ws, hipStream_t s) {
    DistillParams p = distill_params(logits, rows, V, stride, bf, T, ids, lp, k, tail);
    p.loss = loss;
    p.part = static_cast<float4 *>(ws);
    p.stats = reinterpret_cast<float4 *>(stats);
    hipError_t e = run_distill_slice(bf, p.vps, (unsigned)((int64_t)rows * p.S), p, s);
    if (e != hipSuccess) return e;
    const dim3 grid((rows + kNT / 64 - 1) / (kNT / 64));
    if (bf)
        hipLaunchKernelGGL(distill_join<true>, grid, dim3(kNT), 0, s, p);
    else
        hipLaunchKernelGGL(distill_join<false>, grid, dim3(kNT), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_distill_backward(const void *logits, int rows, int V, int64_t stride, bool bf, float T,
                                   const int32_t *ids, const float *lp, int k, bool tail, const float *stats,
                                   const float *grad, void *out, int64_t out_stride, hipStream_t s) {
    DistillParams p = distill_params(logits, rows, V, stride, bf, T, ids, lp, k, tail);
    p.stats = reinterpret_cast<float4 *>(const_cast<float *>(stats));
    p.grad = grad, p.out = out, p.out_stride = out_stride;
    return run_distill_grad(bf, p.vps, (unsigned)((int64_t)rows * p.S), p, s);
}

hipError_t launch_distill_grad(const void *logits, int rows, int V, int64_t stride, bool bf, float T,
                               const int32_t *ids, const float *lp, int k, bool tail, const float *grad, float *loss,
                               void *out, int64_t out_stride, void *ws, hipStream_t s) {
    const int epv = bf ? 8 : 4, nv = V / epv;
    const bool even = V % epv == 0 && stride % epv == 0 && out_stride % epv == 0 &&
                      ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    if (even && nv <= kWholeMax && (nv >= kWholeMin || rows <= kWholeRows)) {
        DistillParams p = distill_params(logits, rows, V, stride, bf, T, ids, lp, k, tail);
        p.loss = loss, p.grad = grad, p.out = out, p.out_stride = out_stride;
        return run_distill_rows(bf, nv, p, s);
    }
    int S, vps;
    cut(rows, V, bf, &S, &vps);
    float *stats = reinterpret_cast<float *>(static_cast<char *>(ws) + up256((int64_t)rows * S * sizeof(float4)));
    hipError_t e = launch_distill_forward(logits, rows, V, stride, bf, T, ids, lp, k, tail, loss, stats, ws, s);
    if (e != hipSuccess) return e;
    return launch_distill_backward(logits, rows, V, stride, bf, T, ids, lp, k, tail, stats, grad, out, out_stride, s);
}

}  // namespace mil
