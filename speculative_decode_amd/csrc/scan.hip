// The layer as a differentiable scan over whole sequences: forward from any initial state,
// and the gradients of everything that goes into it.  General kernels, for fp32 tokens and
// for the shapes the bf16 matrix-core kernels do not take.
//
// Per (sequence, head), with a_t = sum of dt A over a chunk's tokens up to and including t,
// L(t, s) = e^{a_t - a_s} for s <= t, h the state entering the chunk and Lam the gradient of
// the state leaving it:
//   y_t  = sum_s L(t,s) (C_t.B_s) dt_s x_s + e^{a_t} C_t^T h + D x_t
//   h'   = e^{a_Q} h + sum_s e^{a_Q - a_s} dt_s B_s x_s^T            (state leaving the chunk)
//   Lam' = e^{a_Q} Lam + sum_t e^{a_t} C_t dy_t^T                    (gradient of h)
//   dx_s = dt_s (sum_t L(t,s) (C_t.B_s) dy_t + e^{a_Q - a_s} Lam^T B_s) + D dy_s
//   dB_s = dt_s (sum_t L(t,s) (dy_t.x_s) C_t + e^{a_Q - a_s} Lam x_s)          (summed over heads)
//   dC_t = sum_s L(t,s) (dy_t.x_s) dt_s B_s + e^{a_t} h dy_t                   (summed over heads)
// and with W(t,s) = L(t,s) (C_t.B_s) (dy_t.x_s), E_t = e^{a_t} C_t^T h dy_t,
// F_s = e^{a_Q - a_s} B_s^T Lam x_s, the gradient of the exponent dt_u A is
//   g_u  = sum_{s < u <= t} dt_s W(t,s) + sum_{t >= u} E_t + sum_{s < u} dt_s F_s + e^{a_Q} <Lam, h>
//   ddt_u = A g_u + sum_t W(t,u) + F_u,   dA = sum dt_u g_u,   dD = sum dy.x
// g is a direct sum over the pairs whose path crosses u, not a difference of running sums.
//
// Exponents are fp64 sums over the chunk, so that e^{a_t - a_s} is as exact as its
// difference, however far the sum has run.  Everything else is fp32: the products run on
// v_mfma_f32_16x16x4_f32, whose operands the lanes fetch where they lie, weights applied on
// the way.  A lane takes four neighbouring inner indices for four steps at once, so that
// an operand that is contiguous along them is one 16-byte load; the fetches' latency is
// what bounds these kernels, and up to 16 waves a workgroup share it.
//
// Launches: chunk states, a pass over the chunks that turns them into the states entering
// each, outputs; backward the same in reverse with C and dy in the places of B and x, then
// the gradients, whose sums over the heads of a group and over chunks are made by two more
// launches in a fixed order: results do not depend on timing.
#include "scan.h"

namespace mil {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool BF>
__device__ __forceinline__ float tok(const void *p, int64_t i) {
    if constexpr (BF)
        return __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(p)[i] << 16);
    else
        return reinterpret_cast<const float *>(p)[i];
}
template <bool BF>
__device__ __forceinline__ void put(void *p, int64_t i, float v) {
    if constexpr (BF)
        reinterpret_cast<__bf16 *>(p)[i] = (__bf16)v;
    else
        reinterpret_cast<float *>(p)[i] = v;
}

// four token values from element i (a multiple of 4) on
template <bool BF>
__device__ __forceinline__ f32x4 tok4(const void *p, int64_t i) {
    if constexpr (BF) {
        const uint2 w = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p) + i);
        return (f32x4){__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                       __uint_as_float(w.y & 0xffff0000u)};
    } else {
        return *reinterpret_cast<const f32x4 *>(reinterpret_cast<const float *>(p) + i);
    }
}
// f(k), f(k + 1), f(k + 2), f(k + 3)
template <typename F>
__device__ __forceinline__ f32x4 each4(int k, F f) {
    return (f32x4){f(k), f(k + 1), f(k + 2), f(k + 3)};
}
// One 16 x 16 tile of a product over k = 0 .. K-1 (K a multiple of 16): a(i, k) gives A's row i at
// inner indices k .. k + 3, b(k, j) B's column j.  Result register r of lane l is element
// (4 (l / 16) + r, l % 16).
template <typename FA, typename FB>
__device__ __forceinline__ f32x4 tile(int K, FA a, FB b) {
    const int l = threadIdx.x & 63, i = l & 15, kk = 4 * (l >> 4);
    f32x4 acc = {};
#pragma unroll 2
    for (int k = 0; k < K; k += 16) {
        const f32x4 x = a(i, k + kk), y = b(k + kk, i);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], y[e], acc, 0, 0, 0);
    }
    return acc;
}

constexpr int kQ = kScanGeneralChunk;  // 64 tokens: one wave scans a chunk's exponents

// The chunk a workgroup works on.
struct Chunk {
    int seq, c, h, g, len;  // len: live tokens of this chunk (0 .. kQ)
    int64_t t0;             // first token, counted over all sequences
};
__device__ __forceinline__ Chunk chunk_of(const ScanParams &p, int64_t item) {
    Chunk k;
    k.h = (int)(item % p.H);
    k.c = (int)(item / p.H % p.nch);
    k.seq = (int)(item / p.H / p.nch);
    k.g = k.h / (p.H / p.G);
    const int live = scan_length(p, k.seq);
    k.len = max(0, min(kQ, live - k.c * kQ));
    k.t0 = (int64_t)k.seq * p.T + (int64_t)k.c * kQ;
    return k;
}
// a[t] (inclusive) and dt[t] of a chunk, zero dt behind its live tokens.
template <bool BF>
__device__ __forceinline__ void exponents(const ScanParams &p, const Chunk &k, double *a, float *dts) {
    const int t = threadIdx.x;
    if (t < kQ) {
        const float d = t < k.len ? tok<BF>(p.dt, (k.t0 + t) * p.H + k.h) : 0.f;
        double v = (double)d * (double)p.A[k.h];
        if (t >= k.len) v = 0.0;
        if (v < kScanForgets) v = kScanForgets;
#pragma unroll
        for (int s = 1; s < kQ; s <<= 1) {
            const double o = __shfl_up(v, s);
            if (t >= s) v += o;
        }
        a[t] = v;
        dts[t] = d;
    }
    __syncthreads();
}
__device__ __forceinline__ float grow(double e) { return expf((float)e); }

// Chunk states: sum_s w_s u_s v_s^T, [N][P].  Forward: u = B, v = x, w_s = dt_s e^{a_Q - a_s};
// backward: u = C, v = dy, w_t = e^{a_t}.  One workgroup per chunk, head and 64 rows of N.
// (Figures here and below: fp32, 2 sequences of 777 tokens, 8 heads of 64 x 64, 208 workgroups.)
// 11 to 12.5 us.
template <bool BF, bool BACK>
__global__ __launch_bounds__(1024) void scan_part(const ScanParams p) {
    __shared__ double a[kQ];
    __shared__ float dts[kQ], w[kQ];
    const int slabs = (p.N + 63) / 64;
    const Chunk k = chunk_of(p, blockIdx.x / slabs);
    const int n0 = (int)(blockIdx.x % slabs) * 64, nt = min(64, p.N - n0) / 16, pt = p.P / 16;
    exponents<BF>(p, k, a, dts);
    if (threadIdx.x < kQ) {
        const int s = threadIdx.x;
        w[s] = BACK ? grow(a[s]) : dts[s] * grow(a[kQ - 1] - a[s]);
        if (!BACK && n0 == 0 && s == 0) p.total[(int64_t)blockIdx.x / slabs] = a[kQ - 1];
    }
    __syncthreads();
    const void *u = BACK ? p.C : p.B, *v = BACK ? p.dy : p.x;
    const int64_t su = (int64_t)p.G * p.N, sv = (int64_t)p.H * p.P;
    const int64_t bu = k.t0 * su + (int64_t)k.g * p.N, bv = k.t0 * sv + (int64_t)k.h * p.P;
    float *out = (BACK ? p.lam : p.states) + ((int64_t)blockIdx.x / slabs) * p.N * p.P;
    const int lane = threadIdx.x & 63, K = (k.len + 15) / 16 * 16, nw = blockDim.x >> 6;
    for (int q = threadIdx.x >> 6; q < nt * pt; q += nw) {
        const int n = n0 + q / pt * 16, c = q % pt * 16;
        const f32x4 r = tile(
            K,
            [&](int i, int s0) {
                return each4(s0, [&](int s) { return s < k.len ? w[s] * tok<BF>(u, bu + s * su + n + i) : 0.f; });
            },
            [&](int s0, int j) {
                return each4(s0, [&](int s) { return s < k.len ? tok<BF>(v, bv + s * sv + c + j) : 0.f; });
            });
#pragma unroll
        for (int e = 0; e < 4; ++e) out[(int64_t)(n + 4 * (lane >> 4) + e) * p.P + c + (lane & 15)] = r[e];
    }
}

// The states entering each chunk (BACK: the gradients of the states leaving it), in place
// of the chunks' own contributions; one thread per state element.
template <bool BACK>
__global__ __launch_bounds__(256) void scan_pass(const ScanParams p) {
    const int64_t NP = (int64_t)p.N * p.P;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= (int64_t)p.nseq * p.H * NP) return;
    const int64_t sh = at / NP, e = at % NP;
    const int seq = (int)(sh / p.H), h = (int)(sh % p.H);
    const float *from = BACK ? p.dhT : p.h0;
    float *to = BACK ? p.dh0 : p.hT, *buf = BACK ? p.lam : p.states;
    float cur = from ? from[at] : 0.f;
    for (int q = 0; q < p.nch; ++q) {
        const int c = BACK ? p.nch - 1 - q : q;
        const int64_t ch = ((int64_t)seq * p.nch + c) * p.H + h;
        const float part = buf[ch * NP + e];
        buf[ch * NP + e] = cur;
        cur = fmaf(grow(p.total[ch]), cur, part);
    }
    if (to) to[at] = cur;
}

// y of a chunk: one workgroup per chunk and head.  13 us.
template <bool BF>
__global__ __launch_bounds__(1024) void scan_out(const ScanParams p) {
    __shared__ double a[kQ];
    __shared__ float dts[kQ];
    __shared__ __align__(16) float M[kQ][kQ + 4];
    const Chunk k = chunk_of(p, blockIdx.x);
    exponents<BF>(p, k, a, dts);
    const int64_t sn = (int64_t)p.G * p.N, sp = (int64_t)p.H * p.P;
    const int64_t bn = k.t0 * sn + (int64_t)k.g * p.N, bp = k.t0 * sp + (int64_t)k.h * p.P;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r0 = 4 * (lane >> 4), j = lane & 15;
    const int rows = (k.len + 15) / 16, nw = blockDim.x >> 6;
    auto rowC = [&](int t, int n) { return t < k.len ? tok4<BF>(p.C, bn + t * sn + n) : f32x4{}; };
    auto rowB = [&](int s, int n) { return s < k.len ? tok4<BF>(p.B, bn + s * sn + n) : f32x4{}; };
    for (int q = wave; q < rows * rows; q += nw) {
        const int t = q / rows * 16, s = q % rows * 16;
        f32x4 r = {};
        if (s <= t)  // later sources: zeros
            r = tile(
                p.N, [&](int i, int n) { return rowC(t + i, n); }, [&](int n, int jj) { return rowB(s + jj, n); });
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tt = t + r0 + e, ss = s + j;
            M[tt][ss] = ss <= tt ? r[e] * grow(a[tt] - a[ss]) * dts[ss] : 0.f;
        }
    }
    __syncthreads();
    const float *h = p.states + (int64_t)blockIdx.x * p.N * p.P;
    const float D = p.D[k.h];
    const int live_rows = (int)min((int64_t)kQ, p.T - (int64_t)k.c * kQ), pt = p.P / 16;
    for (int q = wave; q < (live_rows + 15) / 16 * pt; q += nw) {
        const int t = q / pt * 16, c = q % pt * 16;
        f32x4 in = {}, up = {};
        if (t < k.len) {
            in = tile(
                t + 16, [&](int i, int s) { return *reinterpret_cast<const f32x4 *>(&M[t + i][s]); },
                [&](int s0, int jj) {
                    return each4(s0, [&](int s) { return s < k.len ? tok<BF>(p.x, bp + s * sp + c + jj) : 0.f; });
                });
            up = tile(
                p.N, [&](int i, int n) { return rowC(t + i, n); },
                [&](int n0, int jj) { return each4(n0, [&](int n) { return h[(int64_t)n * p.P + c + jj]; }); });
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tt = t + r0 + e;
            if (tt >= live_rows) continue;
            const int64_t o = bp + tt * sp + c + j;
            put<BF>(p.y, o, tt < k.len ? in[e] + grow(a[tt]) * up[e] + D * tok<BF>(p.x, o) : 0.f);
        }
    }
}

// Gradients of a chunk: one workgroup per chunk and head.  dB and dC go to per-head fp32
// rows; dA and dD to one partial sum each.  38 us (22 for a single chunk of 16 x 16: the chain of
// dependent products and sums; matrix cores 15 % busy, vector ALU 31 %).  With one inner index
// a lane and 4 waves it took 69.
template <bool BF>
__global__ __launch_bounds__(1024) void scan_grad(const ScanParams p) {
    __shared__ double a[kQ];
    __shared__ __align__(16) float dts[kQ];
    __shared__ float SL[kQ][kQ + 1], W[kQ][kQ + 1];
    __shared__ __align__(16) float DL[kQ][kQ + 4];
    __shared__ float sE[kQ][16], sF[kQ][16], sRed[16], sG[kQ];
    __shared__ double sDD[16];
    const Chunk k = chunk_of(p, blockIdx.x);
    exponents<BF>(p, k, a, dts);
    const int64_t sn = (int64_t)p.G * p.N, sp = (int64_t)p.H * p.P, sh = (int64_t)p.H * p.N;
    const int64_t bn = k.t0 * sn + (int64_t)k.g * p.N, bp = k.t0 * sp + (int64_t)k.h * p.P;
    const int64_t bh = k.t0 * sh + (int64_t)k.h * p.N;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r0 = 4 * (lane >> 4), j = lane & 15;
    const int rows = (k.len + 15) / 16, nw = blockDim.x >> 6;
    const double aQ = a[kQ - 1];
    auto tokC = [&](int t, int n) { return t < k.len ? tok<BF>(p.C, bn + t * sn + n) : 0.f; };
    auto tokB = [&](int s, int n) { return s < k.len ? tok<BF>(p.B, bn + s * sn + n) : 0.f; };
    auto tokY = [&](int t, int c) { return t < k.len ? tok<BF>(p.dy, bp + t * sp + c) : 0.f; };
    auto rowC = [&](int t, int n) { return t < k.len ? tok4<BF>(p.C, bn + t * sn + n) : f32x4{}; };
    auto rowB = [&](int s, int n) { return s < k.len ? tok4<BF>(p.B, bn + s * sn + n) : f32x4{}; };
    auto rowX = [&](int s, int c) { return s < k.len ? tok4<BF>(p.x, bp + s * sp + c) : f32x4{}; };
    auto rowY = [&](int t, int c) { return t < k.len ? tok4<BF>(p.dy, bp + t * sp + c) : f32x4{}; };

    // pair tiles; the strictly later sources' places hold zeros
    for (int q = wave; q < rows * rows; q += nw) {
        const int t = q / rows * 16, s = q % rows * 16;
        f32x4 S = {}, dS = {};
        if (s <= t) {
            S = tile(
                p.N, [&](int i, int n) { return rowC(t + i, n); }, [&](int n, int jj) { return rowB(s + jj, n); });
            dS = tile(
                p.P, [&](int i, int c) { return rowY(t + i, c); }, [&](int c, int jj) { return rowX(s + jj, c); });
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tt = t + r0 + e, ss = s + j;
            const float L = ss <= tt ? grow(a[tt] - a[ss]) : 0.f;
            const float sl = ss <= tt ? S[e] * L : 0.f, d = ss <= tt ? dS[e] : 0.f;
            SL[tt][ss] = sl;
            DL[tt][ss] = ss <= tt ? d * L : 0.f;
            W[tt][ss] = sl * d;
        }
    }
    __syncthreads();
    const float *h = p.states + (int64_t)blockIdx.x * p.N * p.P, *lam = p.lam + (int64_t)blockIdx.x * p.N * p.P;
    const float D = p.D[k.h];
    const int have = (int)min((int64_t)kQ, p.T - (int64_t)k.c * kQ), pt = p.P / 16, ntl = p.N / 16;
    const int tiles = (have + 15) / 16;
    float dd = 0.f;
    for (int q = wave; q < tiles * pt; q += nw) {  // dx
        const int s = q / pt * 16, c = q % pt * 16;
        f32x4 in = {}, out = {};
        if (s < k.len) {
            in = tile(
                rows * 16 - s, [&](int i, int t0) { return each4(t0, [&](int t) { return SL[s + t][s + i]; }); },
                [&](int t0, int jj) { return each4(t0, [&](int t) { return tokY(s + t, c + jj); }); });
            out = tile(
                p.N, [&](int i, int n) { return rowB(s + i, n); },
                [&](int n0, int jj) { return each4(n0, [&](int n) { return lam[(int64_t)n * p.P + c + jj]; }); });
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int ss = s + r0 + e;
            if (ss >= have) continue;
            const int64_t o = bp + ss * sp + c + j;
            float v = 0.f;
            if (ss < k.len) {
                const float dyv = tok<BF>(p.dy, o);
                v = dts[ss] * fmaf(grow(aQ - a[ss]), out[e], in[e]) + D * dyv;
                dd = fmaf(dyv, tok<BF>(p.x, o), dd);
            }
            put<BF>(p.dx, o, v);
        }
    }
    for (int q = wave; q < rows * ntl; q += nw) {  // dB and dC, and their parts in E and F
        const int t = q / ntl * 16, n = q % ntl * 16;
        const f32x4 bin = tile(
            rows * 16 - t, [&](int i, int u0) { return each4(u0, [&](int u) { return DL[t + u][t + i]; }); },
            [&](int u0, int jj) { return each4(u0, [&](int u) { return tokC(t + u, n + jj); }); });
        const f32x4 bout = tile(
            p.P, [&](int i, int c) { return rowX(t + i, c); },
            [&](int c, int jj) { return *reinterpret_cast<const f32x4 *>(lam + (int64_t)(n + jj) * p.P + c); });
        const f32x4 cin = tile(
            t + 16,
            [&](int i, int s) {
                return *reinterpret_cast<const f32x4 *>(&DL[t + i][s]) * *reinterpret_cast<const f32x4 *>(dts + s);
            },
            [&](int s0, int jj) { return each4(s0, [&](int s) { return tokB(s, n + jj); }); });
        const f32x4 cup = tile(
            p.P, [&](int i, int c) { return rowY(t + i, c); },
            [&](int c, int jj) { return *reinterpret_cast<const f32x4 *>(h + (int64_t)(n + jj) * p.P + c); });
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int tt = t + r0 + e;
            const bool ok = tt < k.len;
            const float fb = ok ? grow(aQ - a[tt]) * bout[e] : 0.f, ec = ok ? grow(a[tt]) * cup[e] : 0.f;
            if (ok) {
                p.dBh[bh + tt * sh + n + j] = dts[tt] * (bin[e] + fb);
                p.dCh[bh + tt * sh + n + j] = cin[e] + ec;
            }
            float vf = fb * tokB(tt, n + j), ve = ec * tokC(tt, n + j);
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) {
                vf += __shfl_xor(vf, d);
                ve += __shfl_xor(ve, d);
            }
            if (j == 0) sF[tt][n / 16] = vf, sE[tt][n / 16] = ve;
        }
    }
    // <Lam, h>
    float dot = 0.f;
    for (int i = tid; i < p.N * p.P; i += blockDim.x) dot = fmaf(lam[i], h[i], dot);
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        dot += __shfl_xor(dot, d);
        dd += __shfl_xor(dd, d);
    }
    if (lane == 0) sRed[wave] = dot, sDD[wave] = dd;
    __syncthreads();
    dot = 0.f;
    for (int w = 0; w < nw; ++w) dot += sRed[w];
    dot *= grow(aQ);
    // exponent gradients: row t's sources before u, then the targets from u on
    float col = 0.f, e = 0.f, f = 0.f;
    const int t = tid;
    if (t < k.len) {
        for (int u = t; u < k.len; ++u) col += W[u][t];
        for (int n = 0; n < ntl; ++n) e += sE[t][n], f += sF[t][n];
    }
    __syncthreads();
    if (t < k.len) {
        float run = 0.f;
        for (int s = 0; s <= t; ++s) {
            const float v = W[t][s] * dts[s];
            W[t][s] = run;
            run += v;
        }
    }
    __syncthreads();
    if (t < kQ) {
        float g = 0.f;
        if (t < k.len)
            for (int u = t; u < k.len; ++u) g += W[u][t];
        float later = t < k.len ? e : 0.f, before = t < k.len ? f * dts[t] : 0.f;
#pragma unroll
        for (int d = 1; d < kQ; d <<= 1) {
            const float x = __shfl_down(later, d), y = __shfl_up(before, d);
            if (t + d < kQ) later += x;
            if (t >= d) before += y;
        }
        const float upto = __shfl_up(before, 1);  // without the token's own, whatever its size
        g += later + (t > 0 ? upto : 0.f) + dot;
        if (t < have) put<BF>(p.ddt, (k.t0 + t) * p.H + k.h, t < k.len ? fmaf(p.A[k.h], g, col + f) : 0.f);
        sG[t] = t < k.len ? g * dts[t] : 0.f;
    }
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int i = 0; i < k.len; ++i) s += (double)sG[i];
        p.dAp[blockIdx.x] = s;
        double d = 0.0;
        for (int w = 0; w < nw; ++w) d += sDD[w];
        p.dDp[blockIdx.x] = d;
    }
}

// dB and dC of a group: its heads' rows added in order; zeros behind a sequence's end.  5 us.
template <bool BF>
__global__ __launch_bounds__(256) void scan_sum_heads(const ScanParams p) {
    const int64_t n = (int64_t)p.nseq * p.T * p.G * p.N;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n) return;
    const int R = p.H / p.G, e = (int)(at % p.N);
    const int64_t tg = at / p.N, g = tg % p.G, t = tg / p.G;
    float b = 0.f, c = 0.f;
    if ((int)(t % p.T) < scan_length(p, (int)(t / p.T))) {
        const int64_t row = (t * p.H + g * R) * p.N + e;
        for (int r = 0; r < R; ++r) {
            b += p.dBh[row + (int64_t)r * p.N];
            c += p.dCh[row + (int64_t)r * p.N];
        }
    }
    put<BF>(p.dB, at, b);
    put<BF>(p.dC, at, c);
}

// Launches of a call: workgroups and their waves, one per tile of the largest product up to 16
struct Launches {
    int64_t chunks, states;  // chunks of all heads, values of all states
    int slabs, part_waves, waves;
};
Launches launches(const ScanParams &p) {
    Launches l;
    l.chunks = (int64_t)p.nseq * p.nch * p.H;
    l.states = (int64_t)p.nseq * p.H * p.N * p.P;
    l.slabs = (p.N + 63) / 64;
    l.part_waves = min(16, (p.N < 64 ? p.N / 16 : 4) * (p.P / 16));
    l.waves = min(16, kQ / 16 * (p.P > p.N ? p.P : p.N) / 16);
    return l;
}
template <bool BF>
hipError_t forward(const ScanParams &p, hipStream_t s) {
    const Launches l = launches(p);
    hipLaunchKernelGGL((scan_part<BF, false>), dim3((unsigned)(l.chunks * l.slabs)), dim3(64 * l.part_waves), 0, s, p);
    hipLaunchKernelGGL((scan_pass<false>), dim3((unsigned)((l.states + 255) / 256)), dim3(256), 0, s, p);
    hipLaunchKernelGGL((scan_out<BF>), dim3((unsigned)l.chunks), dim3(64 * l.waves), 0, s, p);
    return hipGetLastError();
}
template <bool BF>
hipError_t backward(const ScanParams &p, hipStream_t s) {
    const Launches l = launches(p);
    hipLaunchKernelGGL((scan_part<BF, true>), dim3((unsigned)(l.chunks * l.slabs)), dim3(64 * l.part_waves), 0, s, p);
    hipLaunchKernelGGL((scan_pass<true>), dim3((unsigned)((l.states + 255) / 256)), dim3(256), 0, s, p);
    hipLaunchKernelGGL((scan_grad<BF>), dim3((unsigned)l.chunks), dim3(64 * l.waves), 0, s, p);
    const int64_t n = (int64_t)p.nseq * p.T * p.G * p.N;
    hipLaunchKernelGGL((scan_sum_heads<BF>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, p);
    return hipGetLastError();
}

// dA and dD: a head's partial sums over sequences and chunks (or segments), one workgroup per
// head.  Each thread adds its share in order and the threads are joined in a fixed tree.
__global__ __launch_bounds__(256) void scan_sum_parts(const ScanParams p, int64_t parts) {
    __shared__ double sA[256], sD[256];
    const int h = blockIdx.x, tid = threadIdx.x;
    double a = 0.0, d = 0.0;
    for (int64_t i = tid; i < parts; i += 256) {
        a += p.dAp[i * p.H + h];
        d += p.dDp[i * p.H + h];
    }
    sA[tid] = a, sD[tid] = d;
    __syncthreads();
    for (int n = 128; n; n >>= 1) {
        if (tid < n) sA[tid] += sA[tid + n], sD[tid] += sD[tid + n];
        __syncthreads();
    }
    if (tid == 0) p.dA[h] = (float)sA[0], p.dD[h] = (float)sD[0];
}

int64_t up256(int64_t v) { return (v + 255) / 256 * 256; }
// Regions of a workspace, each on a 256-byte boundary; with no base only the size counts.
struct Carve {
    char *base;
    int64_t at = 0;
    template <typename T>
    T *take(int64_t n) {
        T *r = base ? reinterpret_cast<T *>(base + at) : nullptr;
        at += up256(n * (int64_t)sizeof(T));
        return r;
    }
};
void cut(ScanParams &p, bool fast) {
    if (fast)
        scan_mfma_cut(p);
    else
        p.nch = (p.T + kQ - 1) / kQ;
}
// What the segments of a walk leave for those after them
void carve_segments(ScanParams &p, Carve &c) {
    const int64_t n = p.nseg > 1 ? (int64_t)p.nseq * p.H * p.nsub : 0;
    p.seg = c.take<float>(n * p.N * p.P);
    p.seg_decay = c.take<float>(n);
}
int64_t carve_states(ScanParams &p, bool fast, bool keep, void *states) {
    Carve c{static_cast<char *>(states)};
    const int64_t chunks = (int64_t)p.nseq * p.nch * p.H;
    if (fast) carve_segments(p, c);
    if (keep || !fast) p.states = c.take<float>(chunks * p.N * p.P);
    if (!fast) p.total = c.take<double>(chunks);
    return c.at;
}
int64_t carve_backward(ScanParams &p, bool fast, void *ws) {
    Carve c{static_cast<char *>(ws)};
    const int64_t rows = (int64_t)p.nseq * p.T * p.H * p.N;
    const int64_t parts = (int64_t)p.nseq * p.H * (fast ? p.nseg * p.parts : p.nch);
    if (fast) {
        carve_segments(p, c);
        const int64_t n = p.H * p.parts == p.G ? 0 : (int64_t)p.nseq * p.nch * kScanChunk * p.H * p.parts * p.N * 3;
        p.dBh24 = c.take<uint8_t>(n);
        p.dCh24 = c.take<uint8_t>(n);
        if (n == 0) p.dBh24 = p.dCh24 = nullptr;
        p.ddtp = c.take<float>(p.parts > 1 ? (int64_t)p.nseq * p.T * p.H * p.parts : 0);
    } else {
        p.lam = c.take<float>(parts * p.N * p.P);
        p.dBh = c.take<float>(rows);
        p.dCh = c.take<float>(rows);
    }
    p.dAp = c.take<double>(parts);
    p.dDp = c.take<double>(parts);
    return c.at;
}

}  // namespace

// The matrix-core kernels take every shape and type they have; the choice depends on
// nothing else, so that the backward call finds what the forward call left.
bool scan_launchable(ScanParams p) {
    const bool fast = scan_mfma_supported(p);
    cut(p, fast);
    const Launches l = launches(p);
    const int64_t tokens = (int64_t)p.nseq * p.T;
    const auto larger = [](int64_t a, int64_t b) { return a > b ? a : b; };
    int64_t most;
    if (fast) {
        most = (int64_t)p.nseq * p.H * p.parts * (p.nseg > p.nsub ? p.nseg : p.nsub) * 512;
        most = larger(most, larger(l.states / 4, larger((int64_t)p.nseq * p.nch * p.G * p.N * 16, tokens * p.H)));
    } else {
        most = l.chunks * 64 * larger((int64_t)l.slabs * l.part_waves, l.waves);
        most = larger(most, larger(l.states, tokens * p.G * p.N));
    }
    return most <= 0xffffffffll - 255;
}
int64_t scan_states_bytes(ScanParams p, bool keep) {
    const bool fast = scan_mfma_supported(p);
    cut(p, fast);
    return carve_states(p, fast, keep, nullptr);
}
int64_t scan_backward_workspace_bytes(ScanParams p) {
    const bool fast = scan_mfma_supported(p);
    cut(p, fast);
    return carve_backward(p, fast, nullptr);
}
hipError_t launch_scan_forward(ScanParams p, void *states, bool keep, hipStream_t s) {
    const bool fast = scan_mfma_supported(p);
    cut(p, fast);
    carve_states(p, fast, keep, states);
    if (fast) return scan_mfma_forward(p, keep, s);
    return p.bf ? forward<true>(p, s) : forward<false>(p, s);
}
hipError_t launch_scan_backward(ScanParams p, const void *states, void *ws, hipStream_t s) {
    const bool fast = scan_mfma_supported(p);
    cut(p, fast);
    carve_states(p, fast, true, const_cast<void *>(states));
    carve_backward(p, fast, ws);
    hipError_t e = fast ? scan_mfma_backward(p, s) : p.bf ? backward<true>(p, s) : backward<false>(p, s);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(scan_sum_parts, dim3(p.H), dim3(256), 0, s, p, (int64_t)p.nseq * (fast ? p.nseg * p.parts : p.nch));
    return hipGetLastError();
}

}  // namespace mil
