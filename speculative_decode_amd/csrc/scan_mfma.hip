// The differentiable scan for bf16 tokens on the matrix cores (the formulas are at the top
// of scan.hip; P and N from 32 to 256).
//
// What bounds it is memory: per chunk of 64 tokens and head a state of N P fp32 values
// meets 64 (2 P + 2 N / (heads of a group)) token values.  So a workgroup walks over the
// chunks of one (sequence, head) with the state in its registers and no state of the walk
// goes through memory, apart from the one that training has to keep: the state entering
// each chunk, which the backward walk (chunks in reverse, the state's gradient in
// registers) needs beside that gradient.  Where sequences and heads alone do not fill the
// chip, a sequence is cut into segments: a first launch walks each segment from zero for
// its own sum and decay, a second turns those into the state entering each.
//
// Products run on v_mfma_f32_16x16x32_bf16.  Lane l = 16 q + c of an operand holds row (or
// column) c and 8 of 32 inner indices; of a result, column c and rows 4 q .. 4 q + 3.  The inner
// indices of lane group q are taken as 4 q + v and 16 + 4 q + v (v = 0..3) of each 32, so that
// two result tiles one below the other are, rounded to bf16, an operand of the next product
// with no exchange between lanes.  Every product of the walk is arranged with the lane's own
// column as the token: scalings by e^{a_t} and the like are then one factor per lane.
//
// The state is kept as result tiles with lanes along n and registers along p, a wave owning
// whole columns of n: the operand that contracts p, for dB, dC and the scalar products, with
// nothing summed across waves.  What contracts n (y and dx) reads copies of the state's two
// leading bf16 parts, made in LDS once per chunk, transposed (where LDS has room for one, the
// second part first and then the first in its place).
//
// The columns of p are independent of each other but for sums (dB, dC, ddt, dA), so a head
// whose state is larger than 16384 values is walked as two or more heads of fewer columns: a
// state of that size is 32 registers per lane of 8 waves, which leaves room for the tokens of
// the next chunk on their way.
//
// Rounding: token operands are exact.  The state, its gradient and weighted tokens are
// split into three bf16 parts (all 24 bits) wherever a state or the gradient of a decay
// depends on them: an entry of dA is a long sum of terms of either sign, and two parts left
// it 1e-6 to 4e-6 off.  What only outputs in bf16 depend on is split in two parts (16 bits): the pair
// weights, and the states in y and dx.  (In one part the walks were 7 and 10 % faster, but y and
// dx after a few tokens from a given state 1.4 times as far off as their own rounding.)  dB and dC per
// head are kept to the upper 24 bits of fp32, 16 of them significant, until the group's are summed
// (rounded to bf16 there, the sum was off by 1.4 to 1.6 times its own rounding).
//
// Tokens and pair weights sit in LDS row by row, pieces of 4 columns turned about per row so
// that no read meets a bank twice; the transposed operands (inner index = row) are read with
// ds_read_b64_tr_b16, 16 lanes exchanging 4 rows of 16 columns.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "scan.h"

namespace mil {
namespace {

typedef __bf16 bf16;
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kQ = kScanChunk;  // 64 tokens
constexpr int kT = kQ / 16;     // token tiles of a chunk
constexpr double kLog2e = 1.4426950408889634074;

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float lo_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_half(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){a, b}, bf16x2));
}
// nearest bf16 of each value, and of what that leaves
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pack2(a, b);
    lo = pack2(a - lo_half(hi), b - hi_half(hi));
}
// Two result tiles one below the other as an operand of the next product
__device__ __forceinline__ bf16x8 operand(const f32x4 &a, const f32x4 &b) {
    const u32x4 w = {pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(b[0], b[1]), pack2(b[2], b[3])};
    return __builtin_bit_cast(bf16x8, w);
}
// Two values in three bf16 parts (all 24 bits), smallest first
__device__ __forceinline__ void split3(float a, float b, uint32_t &lo, uint32_t &mid, uint32_t &hi) {
    hi = pack2(a, b);
    split2(a - lo_half(hi), b - hi_half(hi), mid, lo);
}
// An operand in three parts, smallest first
struct Parts {
    bf16x8 part[3];
};
__device__ __forceinline__ Parts parts_of(const f32x4 &a, const f32x4 &b) {
    u32x4 w[3];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const f32x4 &f = i < 2 ? a : b;
        uint32_t x, y, z;
        split3(f[2 * (i & 1)], f[2 * (i & 1) + 1], x, y, z);
        w[0][i] = x, w[1][i] = y, w[2][i] = z;
    }
    Parts p;
#pragma unroll
    for (int e = 0; e < 3; ++e) p.part[e] = __builtin_bit_cast(bf16x8, w[e]);
    return p;
}
// An operand with its inner index along tokens, times a weight per token
__device__ __forceinline__ Parts weigh(bf16x8 v, const f32x4 &wa, const f32x4 &wb) {
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    const f32x4 a = {lo_half(w[0]) * wa[0], hi_half(w[0]) * wa[1], lo_half(w[1]) * wa[2], hi_half(w[1]) * wa[3]};
    const f32x4 b = {lo_half(w[2]) * wb[0], hi_half(w[2]) * wb[1], lo_half(w[3]) * wb[2], hi_half(w[3]) * wb[3]};
    return parts_of(a, b);
}
// sum over the 16 lanes of a group (every lane gets it)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum16(float v) {
    v += dpp<0x128>(v);  // row_ror 8, 4, 2, 1
    v += dpp<0x124>(v);
    v += dpp<0x122>(v);
    v += dpp<0x121>(v);
    return v;
}
// sum over the four lane groups
__device__ __forceinline__ float sum_q(float v) {
    v += __shfl_xor(v, 16);
    v += __shfl_xor(v, 32);
    return v;
}

// Bounded views: what lies behind `bytes` reads as zero and is not written, so rows behind a
// sequence's end need no branch, and addresses are one offset per lane and one per wave.
typedef __amdgpu_buffer_rsrc_t Buf;
__device__ __forceinline__ Buf view(const void *base, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(Buf b, int lane_off, int off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(b, lane_off, off, 0));
}
__device__ __forceinline__ void store4(Buf b, int lane_off, int off, const f32x4 &v) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 w = {pack2(v[0], v[1]), pack2(v[2], v[3])};
    __builtin_amdgcn_raw_buffer_store_b64(w, b, lane_off, off, 0);
}

// Values that are added up once more: rounded to the upper 24 bits of fp32, four of them in 12
// bytes (two words of upper halves, then the third bytes).
__device__ __forceinline__ void store4x24(Buf b, int lane_off, int off, const f32x4 &v) {
    typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __float_as_uint(v[i]) + 0x80;
    const u32x3 w = {__builtin_amdgcn_perm(r[1], r[0], 0x07060302), __builtin_amdgcn_perm(r[3], r[2], 0x07060302),
                     __builtin_amdgcn_perm(r[1], r[0], 0x0c0c0501) | __builtin_amdgcn_perm(r[3], r[2], 0x05010c0c)};
    __builtin_amdgcn_raw_buffer_store_b96(w, b, lane_off, off, 0);
}

// A barrier that waits for LDS alone: everything waves hand each other here goes through it,
// and the loads of the next chunk and the stores of this one stay in flight across it.
__device__ __forceinline__ void barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Instructions are not moved across: keeps one part's operands out of the registers of another
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

// A tile of kQ rows of W bf16 values in LDS, in pieces of 4 (8 bytes).  Piece u of row r sits
// at place u ^ turn(r), which spreads over all banks both the reads of an operand whose
// inner index is the column (16 rows, two pieces each) and the transposed reads of one whose
// inner index is the row (4 neighbouring pieces of 8 rows).  turn is even: 16-byte halves of
// an aligned pair stay together.
template <int W>
struct Rows {
    static constexpr int ELEMS = kQ * W;
    bf16 *p;
    static __device__ __forceinline__ int turn(int r) {
        const int a = W >= 128 ? r & 7 : W == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
        return 4 * a + ((r >> 2) & 2);
    }
    // Byte offsets.  A row is a power of two long, so whatever of a piece's number is known
    // when compiling (or uniform) is turned into the lane's offset by one exclusive or.
    static __device__ __forceinline__ int at(int r, int u) { return r * W * 2 + 8 * (u ^ turn(r)); }
    __device__ __forceinline__ const char *base() const { return reinterpret_cast<const char *>(p); }
    // operand: row r0 + c (r0 a multiple of 16), inner indices 32 k ..  `o` = row_off()
    static __device__ __forceinline__ int row_off() {
        const int l = threadIdx.x & 63;
        return at(l & 15, l >> 4);
    }
    __device__ __forceinline__ bf16x8 row(int o, int r0, int k) const {
        const uint2 x = *reinterpret_cast<const uint2 *>(base() + r0 * W * 2 + (o ^ (64 * k)));
        const uint2 y = *reinterpret_cast<const uint2 *>(base() + r0 * W * 2 + (o ^ (64 * k + 32)));
        return __builtin_bit_cast(bf16x8, (u32x4){x.x, x.y, y.x, y.y});
    }
    // 4 values of row r0 + c from column 4 q + n0 (n0 a multiple of 16)
    __device__ __forceinline__ f32x4 four(int o, int r0, int n0) const {
        const uint2 w = *reinterpret_cast<const uint2 *>(base() + r0 * W * 2 + (o ^ (2 * n0)));
        return (f32x4){lo_half(w.x), hi_half(w.x), lo_half(w.y), hi_half(w.y)};
    }
    __device__ __forceinline__ void put4(int o, int r0, int n0, uint32_t a, uint32_t b) const {
        *reinterpret_cast<uint2 *>(reinterpret_cast<char *>(p) + r0 * W * 2 + (o ^ (2 * n0))) = make_uint2(a, b);
    }
    // operand: column c0 + c (c0 a multiple of 16), inner indices the rows 32 i ..  `o` = col_off()
    static __device__ __forceinline__ int col_off() {
        const int l = threadIdx.x & 63, j = l & 15;
        return at(4 * (l >> 4) + (j >> 2), j & 3);
    }
    __device__ __forceinline__ bf16x8 col(int o, int c0, int i) const {
        const char *a = base() + 64 * i * W + (o ^ (2 * c0));
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(a));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(a + 32 * W));
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        return __builtin_bit_cast(bf16x8, (s16x8){x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]});
    }
};

// a[t] += (three-part operand) x (rows of token tile t, inner indices 32 i ..) for all token tiles
template <int W>
__device__ __forceinline__ void contract(const Rows<W> &rows, int o, int i, const Parts &l, f32x4 (&a)[kT]) {
    bf16x8 x[kT];
#pragma unroll
    for (int t = 0; t < kT; ++t) x[t] = rows.row(o, 16 * t, i);
#pragma unroll
    for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int t = 0; t < kT; ++t) a[t] = mfma(l.part[e], x[t], a[t]);
}

// Token rows on their way from memory to LDS: 16-byte pieces in registers.
template <int W, int THREADS>
struct Stage {
    static constexpr int ALL = kQ * W / 8, PER = (ALL + THREADS - 1) / THREADS;
    static_assert(ALL % THREADS == 0 || PER == 1, "whole rounds, or one that some threads sit out");
    static constexpr int STEP = THREADS / (W / 8);  // rows a round covers
    u32x4 v[PER];
    // b: the chunk's rows, `stride` bytes apart, bounded to the live ones
    __device__ __forceinline__ void load(Buf b, int stride) {
        const int r = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8);
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = load16(b, r * stride + 16 * c, i * STEP * stride);
    }
    __device__ __forceinline__ void store(const Rows<W> &t) const {
        const int r = threadIdx.x / (W / 8), c = threadIdx.x % (W / 8);
        if (ALL % THREADS != 0 && (int)threadIdx.x >= ALL) return;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            *reinterpret_cast<u32x4 *>(reinterpret_cast<char *>(t.p) + Rows<W>::at(r + i * STEP, 2 * c)) = v[i];
    }
};

// Per-token scalars of a chunk.  a_t in units of log 2, fp64 sums kept as hi + lo, so that a
// difference is as exact as itself.
struct Scalars {
    float hi[kQ], lo[kQ], dt[kQ], up[kQ], down[kQ];  // up = e^{a_t}, down = e^{a_Q - a_t}
};
// By one wave; raw: this lane's dt (0 behind the chunk's end).  Returns the chunk's exponent.
__device__ __forceinline__ double fill_scalars(Scalars &s, uint16_t raw, float A) {
    const int t = threadIdx.x & 63;
    const float d = lo_half(raw);
    double v = (double)d * ((double)A * kLog2e);
    if (d == 0.f) v = 0.0;
    if (v < kScanForgets) v = kScanForgets;
#pragma unroll
    for (int k = 1; k < kQ; k <<= 1) {
        const double o = __shfl_up(v, k);
        if (t >= k) v += o;
    }
    const double all = __shfl(v, kQ - 1);
    const float h = (float)v;
    s.hi[t] = h;
    s.lo[t] = (float)(v - (double)h);
    s.dt[t] = d;
    s.up[t] = __builtin_amdgcn_exp2f((float)v);
    s.down[t] = __builtin_amdgcn_exp2f((float)(all - v));
    return all;
}
__device__ __forceinline__ f32x4 four(const float *p) { return *reinterpret_cast<const f32x4 *>(p); }

// What a workgroup walks over: columns [v P', (v + 1) P') of head h
struct Walk {
    int seq, h, v, g, seg, c0, c1, live;  // chunks [c0, c1); live tokens of the sequence
    int64_t tok0;
};
__device__ __forceinline__ Walk walk_of(const ScanParams &p, int nseg, int segc) {
    // consecutive items (the heads of a group, which share B and C) on one XCD
    const int HV = p.H * p.parts, n = p.nseq * HV * nseg, b = blockIdx.x;
    const int item = n % 8 == 0 ? (b % 8) * (n / 8) + b / 8 : b;
    Walk w;
    w.v = item % p.parts;
    w.h = item % HV / p.parts;
    w.seg = item / HV % nseg;
    w.seq = item / HV / nseg;
    w.g = w.h / (p.H / p.G);
    w.c0 = min(p.nch, w.seg * segc);
    w.c1 = min(p.nch, w.c0 + segc);
    w.live = scan_length(p, w.seq);
    w.tok0 = (int64_t)w.seq * p.T;
    return w;
}
// dt of this lane's token as it is stored (converting it would wait for it)
__device__ __forceinline__ uint16_t load_dt(const ScanParams &p, const Walk &w, int c) {
    const int stride = p.H * 2, len = max(0, min(kQ, w.live - c * kQ));
    const Buf b = view(static_cast<const char *>(p.dt) + (w.tok0 + (int64_t)c * kQ) * stride + 2 * w.h,
                       (int64_t)(len - 1) * stride + 2);
    return len > 0 ? __builtin_amdgcn_raw_buffer_load_b16(b, (threadIdx.x & 63) * stride, 0, 0) : (uint16_t)0;
}

// Waves of a workgroup: one per 16 columns of n, up to 8
template <int N>
constexpr int waves() {
    return N >= 128 ? 8 : 4;
}
// 16 columns of n of a state [N][stride], from n0 and p0, as result tiles (tile i: rows p 16 i ..)
template <int P>
__device__ __forceinline__ void get_state(const float *s, int stride, int n0, f32x4 (&acc)[P / 16]) {
    const int l = threadIdx.x & 63;
    const float *row = s + (int64_t)(n0 + (l & 15)) * stride + 4 * (l >> 4);
#pragma unroll
    for (int i = 0; i < P / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] = row[16 * i + r];
}
template <int P>
__device__ __forceinline__ void put_state(float *s, int stride, int n0, const f32x4 (&acc)[P / 16]) {
    const int l = threadIdx.x & 63;
    float *row = s + (int64_t)(n0 + (l & 15)) * stride + 4 * (l >> 4);
#pragma unroll
    for (int i = 0; i < P / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) row[16 * i + r] = acc[i][r];
}
// acc = e^{a_Q} acc + sum over the chunk's tokens of (rows' tokens) x (this lane's column's
// tokens, weighted); `u` gives the rows, `v` the columns from c0
template <int R, int WU, int WV>
__device__ __forceinline__ void advance(const Rows<WU> &u, const Rows<WV> &v, int uo, int vo, int c0, float decay,
                                        const f32x4 (&w)[4], f32x4 (&acc)[R / 16]) {
    Parts vw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) vw[i] = weigh(v.col(vo, c0, i), w[2 * i], w[2 * i + 1]);
#pragma unroll
    for (int t = 0; t < R / 16; t += 2)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bf16x8 x = u.col(uo, 16 * t, i), y = u.col(uo, 16 * t + 16, i);
            if (i == 0) acc[t] *= decay, acc[t + 1] *= decay;
#pragma unroll
            for (int e = 0; e < 3; ++e) {
                acc[t] = mfma(x, vw[i].part[e], acc[t]);
                acc[t + 1] = mfma(y, vw[i].part[e], acc[t + 1]);
            }
        }
}
// a token weight per inner index of an operand along tokens, for both 32-token steps
__device__ __forceinline__ void token_weights(const float *a, f32x4 (&w)[4]) {
    const int q = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = four(a + 16 * i + 4 * q);
}

// ---------------------------------------------------------------- segments
// The own contribution to the state (BACK: to its gradient), [N][P], and the whole exponent
// of each sub-segment (a segment, or a half: this launch is light enough for two workgroups
// on a compute unit).  8192 tokens, 32 heads of 128 x 128: 41 us, 79 MB read at 1.9 TB/s; LDS
// (51 %) and vector ALU (48 %) take turns with the matrix cores (36 %).
template <int P, int N, bool BACK>
__global__ __launch_bounds__(waves<N>() * 64) void scan_segments(const ScanParams p) {
    constexpr int NW = waves<N>(), TH = NW * 64, NC = (N / 16 + NW - 1) / NW;
    extern __shared__ __align__(16) char lds[];
    Scalars *sc = reinterpret_cast<Scalars *>(lds);  // [2]
    const Rows<N> u{reinterpret_cast<bf16 *>(sc + 2)};
    const Rows<P> v{u.p + Rows<N>::ELEMS};
    const Walk w = walk_of(p, p.nsub, p.subc);
    if (BACK ? w.seg == 0 : w.seg == p.nsub - 1) return;  // nothing follows it
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int su = p.G * N * 2, sv = p.H * p.P * 2;  // bytes from a token's row to the next
    const char *U = static_cast<const char *>(BACK ? p.C : p.B) + w.tok0 * su + w.g * N * 2;
    const char *V = static_cast<const char *>(BACK ? p.dy : p.x) + w.tok0 * sv + (w.h * p.P + w.v * P) * 2;
    const int uo = Rows<N>::col_off(), vo = Rows<P>::col_off();
    const float A = p.A[w.h];
    f32x4 acc[NC][P / 16] = {};
    double total = 0.0;
    Stage<N, TH> lu;
    Stage<P, TH> lv;
    uint16_t dt = 0;
    const int steps = w.c1 - w.c0;
    auto fetch = [&](int k) {
        const int c = BACK ? w.c1 - 1 - k : w.c0 + k, len = max(0, min(kQ, w.live - c * kQ));
        lu.load(view(U + (int64_t)c * kQ * su, (int64_t)len * su), su);
        lv.load(view(V + (int64_t)c * kQ * sv, (int64_t)len * sv), sv);
        if (wave == 0) dt = load_dt(p, w, c);
    };
    fetch(0);
    for (int k = 0; k < steps; ++k) {
        Scalars &s = sc[k & 1];
        lu.store(u);
        lv.store(v);
        if (wave == 0) {
            total += fill_scalars(s, dt, A);
            if (!BACK) s.down[threadIdx.x] *= s.dt[threadIdx.x];
        }
        barrier();
        if (k + 1 < steps) fetch(k + 1);
        f32x4 wt[4];
        token_weights(BACK ? s.up : s.down, wt);
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if ((wave + i * NW) * 16 < N) advance<P>(v, u, vo, uo, (wave + i * NW) * 16, s.up[kQ - 1], wt, acc[i]);
        barrier();
    }
    const int64_t at = ((int64_t)w.seq * p.H + w.h) * p.nsub + w.seg;
#pragma unroll
    for (int i = 0; i < NC; ++i)
        if ((wave + i * NW) * 16 < N)
            put_state<P>(p.seg + at * N * p.P + w.v * P, p.P, (wave + i * NW) * 16, acc[i]);
    if (threadIdx.x == 0 && w.v == 0) p.seg_decay[at] = (float)exp2(total);
}

// The state entering each segment (BACK: the gradient of the one leaving it), in place of the
// segments' own contributions; one thread per 4 state values.  16 sub-segments of 32 heads of
// 128 x 128: 11 to 12 us, 48 MB at 4.2 TB/s.
template <bool BACK>
__global__ __launch_bounds__(256) void scan_fold(const ScanParams p) {
    const int64_t NP4 = (int64_t)p.N * p.P / 4;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= (int64_t)p.nseq * p.H * NP4) return;
    const int64_t sh = at / NP4, e = at % NP4;
    const float *from = BACK ? p.dhT : p.h0;
    f32x4 cur = {};
    if (from)
        for (int r = 0; r < 4; ++r) cur[r] = from[at * 4 + r];
    const int per = p.segc / p.subc;
    f32x4 *x = reinterpret_cast<f32x4 *>(p.seg) + sh * p.nsub * NP4 + e;
    for (int k0 = 0; k0 < p.nsub; k0 += 8) {
        f32x4 own[8];  // loaded together: one after another would wait for each
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k0 + i;  // (nothing was left for the last, nor is anything asked of it)
            own[i] = k < p.nsub - 1 ? x[(BACK ? p.nsub - 1 - k : k) * NP4] : (f32x4){};
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k0 + i, j = BACK ? p.nsub - 1 - k : k;
            if (k >= p.nsub) break;
            // a segment is entered at its first sub-segment, from behind at its last
            if (BACK ? (j + 1) % per == 0 || k == 0 : j % per == 0) x[j * NP4] = cur;
            if (k < p.nsub - 1) cur = cur * p.seg_decay[sh * p.nsub + j] + own[i];
        }
    }
}

// The state a walk starts from
template <int P, int N, int NC>
__device__ __forceinline__ void enter(const ScanParams &p, const Walk &w, int wave, int back, const float *given,
                                      f32x4 (&acc)[NC][P / 16]) {
    const int64_t sh = (int64_t)w.seq * p.H + w.h;
    const int per = p.segc / p.subc, sub = min((w.seg + back) * per - back, p.nsub - 1);
    const float *s = p.nseg > 1 ? p.seg + (sh * p.nsub + sub) * N * p.P : given ? given + sh * N * p.P : nullptr;
    if (!s) return;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int n0 = (wave + i * waves<N>()) * 16;
        if (n0 < N) get_state<P>(s + w.v * P, p.P, n0, acc[i]);
    }
}
// and leaves
template <int P, int N, int NC>
__device__ __forceinline__ void leave(const ScanParams &p, const Walk &w, int wave, float *to,
                                      const f32x4 (&acc)[NC][P / 16]) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int n0 = (wave + i * waves<N>()) * 16;
        if (n0 < N) put_state<P>(to + ((int64_t)w.seq * p.H + w.h) * N * p.P + w.v * P, p.P, n0, acc[i]);
    }
}
// The pair tiles with s <= t, one after another: (0, 0) (1, 0) (1, 1) (2, 0) ..; t of tile i
__device__ __forceinline__ int tile_t(int i) { return i < 1 ? 0 : i < 3 ? 1 : i < 6 ? 2 : 3; }

// Which 16 x 16 tiles of an output [token][p] a wave makes: PT tiles of p from its first on (NW
// apart or one), TT tiles of tokens from t0 on
template <int P, int N>
struct Tiles {
    static constexpr int NW = waves<N>(), ALL = P / 16 * kT / NW;  // tiles per wave
    static_assert(ALL >= 1, "a tile for every wave");
    static constexpr int TT = ALL < kT ? ALL : kT, PT = ALL / TT;
    static __device__ __forceinline__ int p0(int wave, int i) { return 16 * ((PT > 1 ? wave + i * NW : wave) % (P / 16)); }
    static __device__ __forceinline__ int t0(int wave) { return TT < kT ? wave / (P / 16) * TT : 0; }
};

// The first or second bf16 part of a state held as result tiles, as rows n for what contracts n
template <int P, int N, int NC>
__device__ __forceinline__ void put_part(const Rows<P> &to, int o, int wave, bool second, const f32x4 (&h)[NC][P / 16]) {
#pragma unroll
    for (int k = 0; k < NC; ++k) {
        const int nt = wave + k * waves<N>();
        if (nt * 16 >= N) continue;
#pragma unroll
        for (int i = 0; i < P / 16; ++i) {
            uint32_t h0, l0, h1, l1;
            split2(h[k][i][0], h[k][i][1], h0, l0);
            split2(h[k][i][2], h[k][i][3], h1, l1);
            to.put4(o, 16 * nt, 16 * i, second ? l0 : h0, second ? l1 : h1);
        }
    }
}
// a += (columns of p of a part, or of two) x (rows of tokens), for the wave's own tiles
template <int P, int N, bool TWO>
__device__ __forceinline__ void times_state(const Rows<P> &h, const Rows<P> &low, const Rows<N> &rows, int ho, int o,
                                            int wave, f32x4 (&a)[Tiles<P, N>::PT][Tiles<P, N>::TT]) {
    typedef Tiles<P, N> Own;
#pragma unroll
    for (int u = 0; u < Own::PT; ++u)
#pragma unroll 4
        for (int k = 0; k < N / 32; ++k) {
            const bf16x8 x = h.col(ho, Own::p0(wave, u), k), y = TWO ? low.col(ho, Own::p0(wave, u), k) : x;
#pragma unroll
            for (int t = 0; t < Own::TT; ++t) {
                const bf16x8 r = rows.row(o, 16 * (Own::t0(wave) + t), k);
                if constexpr (TWO) a[u][t] = mfma(y, r, a[u][t]);
                a[u][t] = mfma(x, r, a[u][t]);
            }
        }
}

// ---------------------------------------------------------------- forward
// The state's two parts have a place in LDS each, or take one in turn, the second first, where a compute unit
// then has room for one workgroup more.  In turn costs a barrier a chunk and reads B and C once for each
// part: 8192 tokens, 32 heads of 128 x 128, where nothing is won, 135 us against 122; 16 sequences of 1024 tokens,
// 32 heads of 64 x 128, without states left behind, 131 us against 147.
template <int P, int N>
constexpr size_t lds_forward(int places) {
    return 2 * sizeof(Scalars) + (2 * Rows<kQ>::ELEMS + 2 * Rows<N>::ELEMS + Rows<P>::ELEMS + places * N * P) * 2;
}
// Workgroups to a compute unit: with 128 columns the registers leave room for two, with fewer for four.  (64 x 128
// spills one or two registers a lane for its second one; with less unrolling none, but 1 to 2 % slower.)
template <int P, int N>
constexpr int groups(int places) {
    const int n = (int)(160 * 1024 / lds_forward<P, N>(places)), most = P == 128 ? 2 : 4;
    return n < most ? n : most;
}
template <int P, int N>
constexpr int places() {
    return groups<P, N>(1) > groups<P, N>(2) ? 1 : 2;
}

// KEEP: leave the state entering each chunk behind for the backward walk, as the tiles it is held
// in: [n tile][p tile][lane][4].
// 8192 tokens, 32 heads of 128 x 128 (60 GFLOP with its backward call): 113 us, 122 with the
// states left behind (456 MB at 3.7 TB/s; unit by unit LDS 49 %, vector ALU 44 %, matrix cores
// 22 % busy).  What bounds it is that a chunk's phases follow one another: with 131 KB of LDS one
// workgroup of two waves a SIMD has the compute unit.  (Narrower walks, two of which fit, would
// read B and C and form the pairs once more each; not measured.)
template <int P, int N, bool KEEP>
__global__ __launch_bounds__(waves<N>() * 64, (waves<N>() / 4 * groups<P, N>(places<P, N>()))) void scan_walk(
    const ScanParams p) {
    constexpr bool TURN = places<P, N>() == 1;
    constexpr int NW = waves<N>(), TH = NW * 64, NC = (N / 16 + NW - 1) / NW;
    typedef Tiles<P, N> Own;
    extern __shared__ __align__(16) char lds[];
    Scalars *sc = reinterpret_cast<Scalars *>(lds);
    // pair weights in two parts: row t, column s
    const Rows<kQ> M{reinterpret_cast<bf16 *>(sc + 2)}, ML{M.p + Rows<kQ>::ELEMS};
    const Rows<N> B{ML.p + Rows<kQ>::ELEMS}, C{B.p + Rows<N>::ELEMS};
    const Rows<P> X{C.p + Rows<N>::ELEMS};
    const Rows<P> Hs{X.p + Rows<P>::ELEMS}, Hl{TURN ? Hs.p : Hs.p + N * P};  // the state's parts, row n
    const Walk w = walk_of(p, p.nseg, p.segc);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, q = lane >> 4, c = lane & 15;
    const int sn = p.G * N * 2, sp = p.H * p.P * 2;  // bytes from a token's row to the next
    const int64_t bn = w.tok0 * sn + w.g * N * 2, bp = w.tok0 * sp + (w.h * p.P + w.v * P) * 2;
    const char *gB = static_cast<const char *>(p.B) + bn, *gC = static_cast<const char *>(p.C) + bn;
    const char *gX = static_cast<const char *>(p.x) + bp;
    char *gY = static_cast<char *>(p.y) + bp;
    int ro_n = Rows<N>::row_off(), ro_p = Rows<P>::row_off(), ro_q = Rows<kQ>::row_off();
    int co_n = Rows<N>::col_off(), co_p = Rows<P>::col_off();
    const float A = p.A[w.h], D = p.D[w.h];
    // tiles of later sources stay zero
    for (int i = tid; i < 2 * Rows<kQ>::ELEMS / 8; i += TH) reinterpret_cast<uint4 *>(M.p)[i] = make_uint4(0, 0, 0, 0);
    barrier();

    f32x4 hn[NC][P / 16] = {};
    enter<P, N, NC>(p, w, wave, 0, p.h0, hn);
    Stage<N, TH> lB, lC;
    Stage<P, TH> lX;
    uint16_t dt = 0;
    auto fetch = [&](int ch) {
        const int len = max(0, min(kQ, w.live - ch * kQ));
        lB.load(view(gB + (int64_t)ch * kQ * sn, (int64_t)len * sn), sn);
        lC.load(view(gC + (int64_t)ch * kQ * sn, (int64_t)len * sn), sn);
        lX.load(view(gX + (int64_t)ch * kQ * sp, (int64_t)len * sp), sp);
    };
    fetch(w.c0);
    if (wave == NW - 1) {
        fill_scalars(sc[w.c0 & 1], load_dt(p, w, w.c0), A);
        if (w.c0 + 1 < w.c1) dt = load_dt(p, w, w.c0 + 1);
    }
    for (int ch = w.c0; ch < w.c1; ++ch) {
        // (see the backward walk)
        asm volatile("" : "+v"(ro_n), "+v"(ro_p), "+v"(ro_q), "+v"(co_n), "+v"(co_p), "+v"(lane));
        q = lane >> 4, c = lane & 15;
        const Scalars &s = sc[ch & 1];
        lB.store(B);
        lC.store(C);
        lX.store(X);
        f32x4 *keep = reinterpret_cast<f32x4 *>(p.states) +
                      ((((int64_t)w.seq * p.nch + ch) * p.H + w.h) * p.parts + w.v) * (N * P / 4) + lane;
        if constexpr (KEEP) {
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < P / 16; ++i)
                    if ((wave + k * NW) * 16 < N) keep[((wave + k * NW) * (P / 16) + i) * 64] = hn[k][i];
        }
        if constexpr (!TURN) put_part<P, N, NC>(Hs, ro_p, wave, false, hn);
        put_part<P, N, NC>(Hl, ro_p, wave, true, hn);
        barrier();
        // next to the pairs, one wave forms the scalars of the next chunk
        if (wave == NW - 1 && ch + 1 < w.c1) fill_scalars(sc[(ch + 1) & 1], dt, A);
        constexpr int PW = NW > 4 ? NW - 1 : NW;
        // pair weights (C_t.B_s) L(t,s) dt_s of the tiles with s <= t; rows s, columns t
        for (int i = wave; i < kT * (kT + 1) / 2 && wave < PW; i += PW) {
            const int tt = tile_t(i), st = i - tt * (tt + 1) / 2;
            f32x4 S = {};
#pragma unroll
            for (int k = 0; k < N / 32; ++k) S = mfma(B.row(ro_n, 16 * st, k), C.row(ro_n, 16 * tt, k), S);
            const f32x4 hs = four(s.hi + 16 * st + 4 * q), ls = four(s.lo + 16 * st + 4 * q),
                        ds = four(s.dt + 16 * st + 4 * q);
            const float ht = s.hi[16 * tt + c], lt = s.lo[16 * tt + c];
            float m[4];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                m[r] = (st < tt || 4 * q + r <= c)
                           ? S[r] * __builtin_amdgcn_exp2f((ht - hs[r]) + (lt - ls[r])) * ds[r]
                           : 0.f;
            uint32_t h0, l0, h1, l1;
            split2(m[0], m[1], h0, l0);
            split2(m[2], m[3], h1, l1);
            M.put4(ro_q, 16 * tt, 16 * st, h0, h1);
            ML.put4(ro_q, 16 * tt, 16 * st, l0, l1);
        }
        // the state's part of y, 16 columns of p, lanes along t
        f32x4 ay[Own::PT][Own::TT] = {};
        if constexpr (TURN) {
            phase();
            times_state<P, N, false>(Hl, Hl, C, co_p, ro_n, wave, ay);
            barrier();
            put_part<P, N, NC>(Hs, ro_p, wave, false, hn);
        }
        barrier();
        if (ch + 1 < w.c1) fetch(ch + 1);
        if (wave == NW - 1 && ch + 2 < w.c1) dt = load_dt(p, w, ch + 2);
        const Buf out = view(gY + (int64_t)ch * kQ * sp, (int64_t)min(kQ, p.T - ch * kQ) * sp);
        const int t0 = Own::t0(wave);
        auto make_y = [&]() {
            times_state<P, N, !TURN>(Hs, Hl, C, co_p, ro_n, wave, ay);
#pragma unroll
            for (int u = 0; u < Own::PT; ++u) {
                const int p0 = Own::p0(wave, u);
                f32x4(&a)[Own::TT] = ay[u];
#pragma unroll
                for (int t = 0; t < Own::TT; ++t) a[t] *= s.up[16 * (t0 + t) + c];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 xt = X.col(co_p, p0, i);
#pragma unroll
                    for (int t = 0; t < Own::TT; ++t)
                        if (t0 + t >= 2 * i) {
                            a[t] = mfma(xt, ML.row(ro_q, 16 * (t0 + t), i), a[t]);
                            a[t] = mfma(xt, M.row(ro_q, 16 * (t0 + t), i), a[t]);
                        }
                }
#pragma unroll
                for (int t = 0; t < Own::TT; ++t)
                    store4(out, c * sp + 8 * q, 16 * (t0 + t) * sp + 2 * p0, a[t] + D * X.four(ro_p, 16 * (t0 + t), p0));
            }
        };
        if (wave < 4) make_y();  // (as dx in the backward walk)
        phase();
        f32x4 wt[4], wd[4];
        token_weights(s.down, wt);
        token_weights(s.dt, wd);
#pragma unroll
        for (int i = 0; i < 4; ++i) wt[i] *= wd[i];
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if ((wave + k * NW) * 16 < N)
                advance<P>(X, B, co_p, co_n, (wave + k * NW) * 16, s.up[kQ - 1], wt, hn[k]);
        phase();
        if (wave >= 4) make_y();
        barrier();
    }
    if (w.seg == p.nseg - 1 && p.hT) leave<P, N, NC>(p, w, wave, p.hT, hn);
}

// ---------------------------------------------------------------- backward
// Scalars that a chunk's waves hand to the one that finishes the exponents' gradients, next to the
// pairs of the chunk after: from the pairs, which make the next ones then, ..
struct Sums {
    float col[kT][kQ];      // sum over the targets of tile i of W(t, s)
    float row[kT][kQ];      // sum over the sources of tile j of dt_s W(t, s), j before t's tile
    float diag[kQ];         // pairs of u's own tile that cross u
};
// .. and from the states
template <int N>
struct Ends {
    float E[N / 16][kQ], F[N / 16][kQ];
    float dot[8];
};

// 8192 tokens, 32 heads of 128 x 128: 259 us, 723 MB at 2.8 TB/s; LDS 51 %, vector ALU 49 %
// and matrix cores 23 % busy, as in the walk forward one after another; 31800 cycles a chunk, of
// which the matrix products alone need 7200.  4 sequences of up to 2001 tokens, 32 heads of
// 128 x 256 in two parts each: 596 us, 1.57 GB at 2.6 TB/s (chunks behind a sequence's end are walked
// like any other, on zeros).  (Two parts instead of three behind the states and dA took 11 us less
// at an earlier stage, but left dA 1e-6 off and more.)
template <int P, int N>
__global__ __launch_bounds__(waves<N>() * 64) void scan_walk_back(const ScanParams p) {
    constexpr int NW = waves<N>(), TH = NW * 64, NC = (N / 16 + NW - 1) / NW;
    typedef Tiles<P, N> Own;
    extern __shared__ __align__(16) char lds[];
    Scalars *sc = reinterpret_cast<Scalars *>(lds);
    Sums *sums = reinterpret_cast<Sums *>(sc + 2);  // [2]
    Ends<N> &ends = *reinterpret_cast<Ends<N> *>(sums + 2);
    // pair weights, row s, column t: of dx, and of dB and dC, in two parts each.  Of each the quarter of
    // rows 32.. and columns ..31 is never read; the three of M, DH and DL hold the quarters that M's second
    // part has: (rows, columns) ..31, ..31; ..31, 32..; 32.., 32..
    const Rows<kQ> M{reinterpret_cast<bf16 *>(&ends + 1)}, DH{M.p + Rows<kQ>::ELEMS}, DL{DH.p + Rows<kQ>::ELEMS};
    auto second = [&](int st, int half) { return half == 0 ? M : st < 2 ? DH : DL; };  // of tile row st
    const Rows<N> B{DL.p + Rows<kQ>::ELEMS}, C{B.p + Rows<N>::ELEMS};
    const Rows<P> X{C.p + Rows<N>::ELEMS}, Y{X.p + Rows<P>::ELEMS}, Ls{Y.p + Rows<P>::ELEMS};
    const Walk w = walk_of(p, p.nseg, p.segc);
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    int lane = tid & 63, q = lane >> 4, c = lane & 15;
    const int HV = p.H * p.parts;
    const int sn = p.G * N * 2, sp = p.H * p.P * 2;  // bytes from a token's row to the next
    const int64_t bn = w.tok0 * sn + w.g * N * 2, bp = w.tok0 * sp + (w.h * p.P + w.v * P) * 2;
    const char *gB = static_cast<const char *>(p.B) + bn, *gC = static_cast<const char *>(p.C) + bn;
    const char *gX = static_cast<const char *>(p.x) + bp, *gY = static_cast<const char *>(p.dy) + bp;
    char *oX = static_cast<char *>(p.dx) + bp;
    const bool whole = !p.dBh24;  // the only walk of its group: dB and dC themselves
    int ro_n = Rows<N>::row_off(), ro_p = Rows<P>::row_off(), ro_q = Rows<kQ>::row_off();
    int co_n = Rows<N>::col_off(), co_p = Rows<P>::col_off(), co_q = Rows<kQ>::col_off();
    const float A = p.A[w.h], D = p.D[w.h];
    // tiles of earlier targets stay zero
    for (int i = tid; i < 3 * Rows<kQ>::ELEMS / 8; i += TH)
        reinterpret_cast<uint4 *>(M.p)[i] = make_uint4(0, 0, 0, 0);
    barrier();

    f32x4 ln[NC][P / 16] = {};
    enter<P, N, NC>(p, w, wave, 1, p.dhT, ln);
    Stage<N, TH> lB, lC;
    Stage<P, TH> lX, lY;
    uint16_t dt = 0;
    auto fetch = [&](int ch) {
        const int len = max(0, min(kQ, w.live - ch * kQ));
        lB.load(view(gB + (int64_t)ch * kQ * sn, (int64_t)len * sn), sn);
        lC.load(view(gC + (int64_t)ch * kQ * sn, (int64_t)len * sn), sn);
        lX.load(view(gX + (int64_t)ch * kQ * sp, (int64_t)len * sp), sp);
        lY.load(view(gY + (int64_t)ch * kQ * sp, (int64_t)len * sp), sp);
    };
    double dA = 0.0, dD = 0.0;
    // du, decay: the chunk's dt of this lane's token and its whole decay
    auto finish = [&](int ch, float du, float decay) {
        const Sums &sm = sums[ch & 1];
        const int have = min(kQ, p.T - ch * kQ);
        // gradient of each token's exponent; lane u, m = its tile
        const int u = lane, m = lane >> 4;
        float e = 0.f, f = 0.f, all = 0.f;
#pragma unroll
        for (int i = 0; i < N / 16; ++i) e += ends.E[i][u], f += ends.F[i][u];
#pragma unroll
        for (int i = 0; i < NW; ++i) all += ends.dot[i];
        const float own = sm.col[m][u];
        float after = 0.f;  // targets in later tiles
        for (int i = m + 1; i < kT; ++i) after += sm.col[i][u];
        const float r0 = m > 0 ? sm.row[0][u] : 0.f, r1 = m > 1 ? sm.row[1][u] : 0.f,
                    r2 = m > 2 ? sm.row[2][u] : 0.f;
        float rs = r0 + r1 + r2, cs = after * du;  // rows: suffix over the tile; columns: prefix before u
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
            const float x = __shfl_down(rs, d), y = __shfl_up(cs, d);
            if (c + d < 16) rs += x;
            if (c >= d) cs += y;
        }
        const float R0 = sum16(r0), R1 = sum16(r1);
        const float cb = __shfl_up(cs, 1);  // without the token's own, whatever its size
        const float t20 = __shfl(R0, 32), t30 = __shfl(R0, 48), t31 = __shfl(R1, 48);
        float g = sm.diag[u] + rs + (c > 0 ? cb : 0.f) + (m == 1 ? t20 + t30 : m == 2 ? t30 + t31 : 0.f);
        float later = e, before = f * du;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const float x = __shfl_down(later, d), y = __shfl_up(before, d);
            if (u + d < 64) later += x;
            if (u >= d) before += y;
        }
        const float bb = __shfl_up(before, 1);
        g += later + (u > 0 ? bb : 0.f) + decay * all;
        const bool live = ch * kQ + u < w.live;
        dA += live ? (double)(g * du) : 0.0;
        if (u < have) {
            const float v = live ? fmaf(A, g, own + after + f) : 0.f;
            const int64_t at = (w.tok0 + ch * kQ + u) * p.H + w.h;
            if (p.parts == 1)
                static_cast<uint16_t *>(p.ddt)[at] = (uint16_t)pack2(v, 0.f);
            else
                p.ddtp[at * p.parts + w.v] = v;
        }
    };
    float last_dt = 0.f, last_decay = 1.f;  // of the chunk that `finish` is due for
    fetch(w.c1 - 1);
    if (wave == NW - 1) {
        fill_scalars(sc[(w.c1 - 1) & 1], load_dt(p, w, w.c1 - 1), A);
        if (w.c1 - 2 >= w.c0) dt = load_dt(p, w, w.c1 - 2);
    }
    for (int ch = w.c1 - 1; ch >= w.c0; --ch) {
        // the offsets change as far as the compiler knows, so that the addresses made from
        // them are made again in each chunk instead of filling registers across all of it
        asm volatile("" : "+v"(ro_n), "+v"(ro_p), "+v"(ro_q), "+v"(co_n), "+v"(co_p), "+v"(co_q), "+v"(lane));
        q = lane >> 4, c = lane & 15;
        const Scalars &s = sc[ch & 1];
        Sums &sm = sums[ch & 1];
        lB.store(B);
        lC.store(C);
        lX.store(X);
        lY.store(Y);
        put_part<P, N, NC>(Ls, ro_p, wave, true, ln);
        barrier();
        f32x4 kept[NC][P / 16];
        {
            const f32x4 *keep = reinterpret_cast<const f32x4 *>(p.states) +
                                ((((int64_t)w.seq * p.nch + ch) * p.H + w.h) * p.parts + w.v) * (N * P / 4) + lane;
#pragma unroll
            for (int k = 0; k < NC; ++k)
#pragma unroll
                for (int i = 0; i < P / 16; ++i)
                    kept[k][i] = keep[(min(wave + k * NW, N / 16 - 1) * (P / 16) + i) * 64];
        }
        // next to the pairs, two waves look after the exponents: one finishes the gradients of
        // the chunk before, one forms the scalars of the next
        if (wave == NW - 1 && ch > w.c0) fill_scalars(sc[(ch - 1) & 1], dt, A);
        if (wave == NW - 2 && ch < w.c1 - 1) finish(ch + 1, last_dt, last_decay);
        constexpr int PW = NW > 4 ? NW - 2 : NW;  // waves that share the pairs
        // pairs: rows t, columns s of the tiles with s <= t
        constexpr int PAIRS = kT * (kT + 1) / 2, PT = (PAIRS + PW - 1) / PW;  // tiles, and a wave's at most
        f32x4 S[PT] = {}, G[PT] = {};
        if (wave < PW) {
#pragma unroll 4
            for (int k = 0; k < N / 32; ++k)
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    const int i = min(wave + j * PW, PAIRS - 1), tt = tile_t(i), st = i - tt * (tt + 1) / 2;
                    S[j] = mfma(C.row(ro_n, 16 * tt, k), B.row(ro_n, 16 * st, k), S[j]);
                }
            phase();
#pragma unroll
            for (int k = 0; k < P / 32; ++k)
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    const int i = min(wave + j * PW, PAIRS - 1), tt = tile_t(i), st = i - tt * (tt + 1) / 2;
                    G[j] = mfma(Y.row(ro_p, 16 * tt, k), X.row(ro_p, 16 * st, k), G[j]);
                }
        }
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = wave + j * PW;
            if (wave >= PW || i >= PAIRS) continue;
            const int tt = tile_t(i), st = i - tt * (tt + 1) / 2;
            const f32x4 ht = four(s.hi + 16 * tt + 4 * q), lt = four(s.lo + 16 * tt + 4 * q);
            const float hs = s.hi[16 * st + c], ls = s.lo[16 * st + c], ds = s.dt[16 * st + c];
            f32x4 m, d, v;
            float col = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool ok = st < tt || c <= 4 * q + r;
                const float L = ok ? __builtin_amdgcn_exp2f((ht[r] - hs) + (lt[r] - ls)) : 0.f;
                const float sl = ok ? S[j][r] * L : 0.f, W = ok ? sl * G[j][r] : 0.f;
                m[r] = sl * ds;
                d[r] = ok ? G[j][r] * L * ds : 0.f;
                col += W;
                v[r] = W * ds;
            }
            uint32_t h0, l0, h1, l1;
            split2(m[0], m[1], h0, l0);
            split2(m[2], m[3], h1, l1);
            M.put4(ro_q, 16 * st, 16 * tt, h0, h1);
            second(st, tt >> 1).put4(ro_q, 32 + 16 * (st & 1), 16 * (tt & 1), l0, l1);
            split2(d[0], d[1], h0, l0);
            split2(d[2], d[3], h1, l1);
            DH.put4(ro_q, 16 * st, 16 * tt, h0, h1);
            DL.put4(ro_q, 16 * st, 16 * tt, l0, l1);
            col = sum_q(col);
            if (q == 0) sm.col[tt][16 * st + c] = col;
            if (st == tt) {
                // pairs s < u <= t of one tile: sums over t >= u, then over s < u
                v[2] += v[3], v[1] += v[2], v[0] += v[1];
                const float a1 = __shfl(v[0], c + 16), a2 = __shfl(v[0], c + 32), a3 = __shfl(v[0], c + 48);
                const float later = q == 0 ? a1 + (a2 + a3) : q == 1 ? a2 + a3 : q == 2 ? a3 : 0.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float g = sum16(c < 4 * q + r ? v[r] + later : 0.f);
                    if (c == 0) sm.diag[16 * tt + 4 * q + r] = g;
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float g = sum16(v[r]);
                    if (c == 0) sm.row[st][16 * tt + 4 * q + r] = g;
                }
            }
        }
        // the states' part of dx, 16 columns of p, lanes along s
        f32x4 ax[Own::PT][Own::TT] = {};
        phase();
        times_state<P, N, false>(Ls, Ls, B, co_p, ro_n, wave, ax);
        barrier();
        put_part<P, N, NC>(Ls, ro_p, wave, false, ln);
        if (wave == NW - 1 && ch - 2 >= w.c0) dt = load_dt(p, w, ch - 2);
        last_dt = s.dt[lane], last_decay = s.up[kQ - 1];
        const int have = min(kQ, p.T - ch * kQ);
        barrier();
        auto make_dx = [&]() {
            const Buf out = view(oX + (int64_t)ch * kQ * sp, (int64_t)have * sp);
            const int t0 = Own::t0(wave);
            times_state<P, N, false>(Ls, Ls, B, co_p, ro_n, wave, ax);
#pragma unroll
            for (int u = 0; u < Own::PT; ++u) {
                const int p0 = Own::p0(wave, u);
                f32x4(&a)[Own::TT] = ax[u];
#pragma unroll
                for (int t = 0; t < Own::TT; ++t) a[t] *= s.down[16 * (t0 + t) + c] * s.dt[16 * (t0 + t) + c];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 yt = Y.col(co_p, p0, i);
#pragma unroll
                    for (int t = 0; t < Own::TT; ++t)
                        if (t0 + t < 2 * i + 2) {
                            a[t] = mfma(yt, second(t0 + t, i).row(ro_q, 32 + 16 * ((t0 + t) & 1), 0), a[t]);
                            a[t] = mfma(yt, M.row(ro_q, 16 * (t0 + t), i), a[t]);
                        }
                }
                float dd = 0.f;
#pragma unroll
                for (int t = 0; t < Own::TT; ++t) {
                    const f32x4 yv = Y.four(ro_p, 16 * (t0 + t), p0), xv = X.four(ro_p, 16 * (t0 + t), p0);
#pragma unroll
                    for (int r = 0; r < 4; ++r) dd = fmaf(yv[r], xv[r], dd);
                    store4(out, c * sp + 8 * q, 16 * (t0 + t) * sp + 2 * p0, a[t] + D * yv);
                }
                dD += (double)dd;
            }
        };
        // two waves share a SIMD; its first and its second make dx at different times, so that
        // one's LDS reads meet the other's matrix products
        if (wave < 4) make_dx();
        phase();
        // dB and dC: rows of the outputs, or tiles for the sum over the group as the lanes hold them
        const int64_t part = (((int64_t)w.seq * p.nch + ch) * HV + w.h * p.parts + w.v) * (N * kQ * 3);
        const int64_t row = bn + (int64_t)ch * kQ * sn;
        const Buf outB = whole ? view(static_cast<char *>(p.dB) + row, (int64_t)have * sn) : view(p.dBh24 + part, N * kQ * 3);
        const Buf outC = whole ? view(static_cast<char *>(p.dC) + row, (int64_t)have * sn) : view(p.dCh24 + part, N * kQ * 3);
        auto put_tile = [&](Buf out, int t, int nt, const f32x4 &v) {
            if (whole)
                store4(out, c * sn + 8 * q, 16 * t * sn + 32 * nt, v);
            else
                store4x24(out, 12 * lane, (nt * kT + t) * 768, v);
        };
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k) {  // dB and dC: 16 columns of n, lanes along s and t
            if (k == NC - 1 && ch > w.c0) fetch(ch - 1);  // (with the last tile: the operands of the others are gone)
            const int nt = wave + k * NW, n0 = nt * 16;
            if (n0 >= N) continue;
            {
                f32x4 a[kT] = {};
#pragma unroll
                for (int i = 0; i < P / 32; ++i) {
                    const Parts l = parts_of(ln[k][2 * i], ln[k][2 * i + 1]);
                    contract(X, ro_p, i, l, a);
                }
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    a[t] *= s.down[16 * t + c];
                    const f32x4 b = B.four(ro_n, 16 * t, n0);
                    const float f = sum_q((a[t][0] * b[0] + a[t][1] * b[1]) + (a[t][2] * b[2] + a[t][3] * b[3]));
                    if (q == 0) ends.F[nt][16 * t + c] = f;
                    a[t] *= s.dt[16 * t + c];
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 ct = C.col(co_n, n0, i);
#pragma unroll
                    for (int t = 0; t < 2 * i + 2; ++t) {
                        a[t] = mfma(ct, DL.row(ro_q, 16 * t, i), a[t]);
                        a[t] = mfma(ct, DH.row(ro_q, 16 * t, i), a[t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < kT; ++t) put_tile(outB, t, nt, a[t]);
            }
            phase();
            {
                f32x4 a[kT] = {};
#pragma unroll
                for (int i = 0; i < P / 32; ++i) {
                    const Parts h = parts_of(kept[k][2 * i], kept[k][2 * i + 1]);
                    contract(Y, ro_p, i, h, a);
                }
#pragma unroll
                for (int t = 0; t < kT; ++t) {
                    a[t] *= s.up[16 * t + c];
                    const f32x4 b = C.four(ro_n, 16 * t, n0);
                    const float e = sum_q((a[t][0] * b[0] + a[t][1] * b[1]) + (a[t][2] * b[2] + a[t][3] * b[3]));
                    if (q == 0) ends.E[nt][16 * t + c] = e;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const bf16x8 bt = B.col(co_n, n0, i);
#pragma unroll
                    for (int t = 2 * i; t < kT; ++t) {
                        a[t] = mfma(bt, DL.col(co_q, 16 * t, i), a[t]);
                        a[t] = mfma(bt, DH.col(co_q, 16 * t, i), a[t]);
                    }
                }
#pragma unroll
                for (int t = 0; t < kT; ++t) put_tile(outC, t, nt, a[t]);
            }
            phase();
            // <Lam, h>: both are held in the same places
#pragma unroll
            for (int i = 0; i < P / 16; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) dot = fmaf(ln[k][i][r], kept[k][i][r], dot);
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) dot += __shfl_xor(dot, d);
        if (lane == 0) ends.dot[wave] = dot;
        phase();
        f32x4 wt[4];
        token_weights(s.up, wt);
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if ((wave + k * NW) * 16 < N)
                advance<P>(Y, C, co_p, co_n, (wave + k * NW) * 16, s.up[kQ - 1], wt, ln[k]);
        phase();
        if (wave >= 4) make_dx();
        barrier();
    }
    if (wave == NW - 2) finish(w.c0, last_dt, last_decay);
    if (w.seg == 0 && p.dh0) leave<P, N, NC>(p, w, wave, p.dh0, ln);
    // this walk's parts of dA and dD
    double *red = reinterpret_cast<double *>(sums);
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        dA += __shfl_xor(dA, d);
        dD += __shfl_xor(dD, d);
    }
    barrier();
    if (lane == 0) red[wave] = dD;
    barrier();
    if (wave == NW - 2 && lane == 0) {  // the wave that has dA
        double d = 0.0;
        for (int i = 0; i < NW; ++i) d += red[i];
        const int64_t at = (((int64_t)w.seq * p.nseg + w.seg) * p.parts + w.v) * p.H + w.h;
        p.dAp[at] = dA;
        p.dDp[at] = d;
    }
}

// dB and dC of a group: its heads' 24-bit tiles added in order, a thread for the 4 values that a
// lane of the walk held; zeros behind a sequence's end.  8192 tokens, 32 heads in 8 groups, N =
// 128: 45 us, 235 MB at 5.2 TB/s.  (In bf16 rows 28 us and the walk 7 us less, but dB and dC
// off by 1.4 to 1.6 times their own rounding; 24 bits as rows of two planes: 40 us, the walk 10 more.)
__global__ __launch_bounds__(256) void scan_sum_heads24(const ScanParams p) {
    const int HV = p.H * p.parts, R = HV / p.G, NT = p.N / 16, tiles = NT * kT;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);  // a wave per tile
    if (at >= (int64_t)p.nseq * p.nch * p.G * tiles) return;
    // neighbouring waves make neighbouring columns: whole lines of the output per workgroup
    const int lane = threadIdx.x & 63, tile = (int)(at % tiles), t = tile / NT, nt = tile % NT;
    const int64_t cg = at / tiles, g = cg % p.G, sc = cg / p.G;
    const int seq = (int)(sc / p.nch), tok = (int)(sc % p.nch) * kQ + 16 * t + (lane & 15);
    const int64_t from = ((sc * HV + g * R) * tiles + nt * kT + t) * 768 + 12 * lane;
    const int64_t to = (((int64_t)seq * p.T + tok) * p.G + g) * p.N + 16 * nt + 4 * (lane >> 4);
    if (tok >= p.T) return;
    f32x4 sum[2] = {};
    if (tok < scan_length(p, seq)) {
#pragma unroll 4
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const uint8_t *src = (which ? p.dCh24 : p.dBh24) + from + (int64_t)r * tiles * 768;
                const uint32_t *v = reinterpret_cast<const uint32_t *>(src);
                const uint32_t a = v[0], b = v[1], low = v[2];
                sum[which][0] += __uint_as_float(__builtin_amdgcn_perm(a, low, 0x0504000c));
                sum[which][1] += __uint_as_float(__builtin_amdgcn_perm(a, low, 0x0706010c));
                sum[which][2] += __uint_as_float(__builtin_amdgcn_perm(b, low, 0x0504020c));
                sum[which][3] += __uint_as_float(__builtin_amdgcn_perm(b, low, 0x0706030c));
            }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which)
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(which ? p.dC : p.dB) + to) =
            make_uint2(pack2(sum[which][0], sum[which][1]), pack2(sum[which][2], sum[which][3]));
}

// ddt of a head walked in parts
__global__ __launch_bounds__(256) void scan_sum_ddt(const ScanParams p) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= (int64_t)p.nseq * p.T * p.H) return;
    float v = 0.f;
    for (int i = 0; i < p.parts; ++i) v += p.ddtp[at * p.parts + i];
    static_cast<uint16_t *>(p.ddt)[at] = (uint16_t)pack2(v, 0.f);
}

template <int P, int N>
constexpr size_t lds_segments() {
    return 2 * sizeof(Scalars) + (Rows<N>::ELEMS + Rows<P>::ELEMS) * 2;
}
template <int P, int N>
constexpr size_t lds_backward() {
    return 2 * sizeof(Scalars) + 2 * sizeof(Sums) + sizeof(Ends<N>) +
           (3 * Rows<kQ>::ELEMS + 2 * Rows<N>::ELEMS + 2 * Rows<P>::ELEMS + N * P) * 2;
}
unsigned sub_grid(const ScanParams &p) { return (unsigned)(p.nseq * p.H * p.parts * p.nsub); }
unsigned fold_grid(const ScanParams &p) {
    return (unsigned)(((int64_t)p.nseq * p.H * p.N * p.P / 4 + 255) / 256);
}
// More LDS than a launch may have by default is asked for once per kernel and device
template <auto KERNEL>
hipError_t launch(unsigned grid, unsigned threads, size_t lds, hipStream_t s, const ScanParams &p) {
    static std::atomic<uint64_t> asked{0};  // devices, one bit each (those behind 63 ask every time)
    if (lds > 64 * 1024) {
        int dev = 0;
        hipError_t e = hipGetDevice(&dev);
        if (e != hipSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (!(asked.load(std::memory_order_relaxed) & bit)) {
            e = hipFuncSetAttribute(reinterpret_cast<const void *>(KERNEL),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
            if (e != hipSuccess) return e;
            asked.fetch_or(bit, std::memory_order_relaxed);
        }
    }
    hipLaunchKernelGGL(KERNEL, dim3(grid), dim3(threads), lds, s, p);
    return hipGetLastError();
}

template <int P, int N>
hipError_t forward(const ScanParams &p, bool keep, hipStream_t s) {
    constexpr size_t lds = lds_forward<P, N>(places<P, N>());
    static_assert(lds <= 160 * 1024 && lds_backward<P, N>() <= 160 * 1024, "LDS of a compute unit");
    const unsigned grid = (unsigned)(p.nseq * p.H * p.parts * p.nseg), th = waves<N>() * 64;
    hipError_t e = hipSuccess;
    if (p.nseg > 1) {
        e = launch<scan_segments<P, N, false>>(sub_grid(p), th, lds_segments<P, N>(), s, p);
        if (e == hipSuccess) e = launch<scan_fold<false>>(fold_grid(p), 256, 0, s, p);
    }
    if (e != hipSuccess) return e;
    return keep ? launch<scan_walk<P, N, true>>(grid, th, lds, s, p)
                : launch<scan_walk<P, N, false>>(grid, th, lds, s, p);
}
template <int P, int N>
hipError_t backward(const ScanParams &p, hipStream_t s) {
    const unsigned grid = (unsigned)(p.nseq * p.H * p.parts * p.nseg), th = waves<N>() * 64;
    hipError_t e = hipSuccess;
    if (p.nseg > 1) {
        e = launch<scan_segments<P, N, true>>(sub_grid(p), th, lds_segments<P, N>(), s, p);
        if (e == hipSuccess) e = launch<scan_fold<true>>(fold_grid(p), 256, 0, s, p);
    }
    if (e == hipSuccess) e = launch<scan_walk_back<P, N>>(grid, th, lds_backward<P, N>(), s, p);
    return e;
}
// Columns of p that a walk takes: all of them up to 128 and to a state of 16384 values.  (Whole heads
// of 128 x 256 would need 207 KB of LDS.  An early form that fitted spilled registers: walk back
// 1345 us, in two parts 936, at 4 sequences of up to 2001 tokens and 32 heads.)
int columns(int P, int N) {
    int c = P < 128 ? P : 128;
    while (c * N > 16384) c /= 2;
    return c;
}
template <typename F>
hipError_t by_shape(int P, int N, F f) {
    auto n = [&](auto pc) {
        switch (N) {
            case 32: return f(pc, std::integral_constant<int, 32>{});
            case 64: return f(pc, std::integral_constant<int, 64>{});
            case 128: return f(pc, std::integral_constant<int, 128>{});
            default:
                if constexpr (decltype(pc)::value <= 64) return f(pc, std::integral_constant<int, 256>{});
                return hipErrorInvalidValue;
        }
    };
    switch (columns(P, N)) {
        case 32: return n(std::integral_constant<int, 32>{});
        case 64: return n(std::integral_constant<int, 64>{});
        default: return n(std::integral_constant<int, 128>{});
    }
}

}  // namespace

// Against the general kernels, bf16, 32 heads of 128 x 128, all kernels of forward and backward:
// 1024 tokens 117 us against 390, 8192 tokens 537 against 3190.  (P or N of 16 would leave half of
// every operand's inner indices empty.)
bool scan_mfma_supported(const ScanParams &p) {
    // (the last: a chunk's rows, of up to 4 parts of a head, stay within the 2 GiB of a bounded view)
    return p.bf && p.P >= 32 && p.N >= 32 && (int64_t)p.H * (p.P > 4 * p.N ? p.P : 4 * p.N) < 1 << 23;
}
// Segments: as many as fill the chip with one workgroup per compute unit, but none shorter
// than two chunks (the launch that prepares them walks every segment but one).  8192 tokens, 32
// heads of 128 x 128: walk back 1599 us in one segment, 808 in two, 422 in four, 265 in eight; walk
// forward 708, 357, 192, 124; the preparing launch 71 us in two segments, 43 in four and 42 in eight,
// with its fold 76, 49 and 54 each way.
void scan_mfma_cut(ScanParams &p) {
    p.nch = (p.T + kQ - 1) / kQ;
    p.parts = p.P / columns(p.P, p.N);
    const int walks = p.nseq * p.H * p.parts;
    int n = walks >= 256 ? 1 : 256 / walks;
    n = n > p.nch / 2 ? p.nch / 2 : n;
    n = n < 1 ? 1 : n;
    p.segc = (p.nch + n - 1) / n;
    p.nseg = (p.nch + p.segc - 1) / p.segc;
    // halves where they are long enough to be worth the larger fold (8 chunks and more: 8192
    // tokens of 32 heads 47 -> 42 us against 8.5 -> 12 us; at 2 chunks, 1024 tokens, 11.7 -> 13.3
    // and 8.3 -> 11.4)
    p.subc = p.segc % 2 == 0 && p.segc >= 8 ? p.segc / 2 : p.segc;
    p.nsub = (p.nch + p.subc - 1) / p.subc;
}
hipError_t scan_mfma_forward(const ScanParams &p, bool keep, hipStream_t s) {
    return by_shape(p.P, p.N, [&](auto P, auto N) { return forward<decltype(P)::value, decltype(N)::value>(p, keep, s); });
}
hipError_t scan_mfma_backward(const ScanParams &p, hipStream_t s) {
    hipError_t e =
        by_shape(p.P, p.N, [&](auto P, auto N) { return backward<decltype(P)::value, decltype(N)::value>(p, s); });
    if (e == hipSuccess && p.H * p.parts > p.G) {
        const int64_t n = (int64_t)p.nseq * p.nch * p.G * (p.N / 16 * kT);
        e = launch<scan_sum_heads24>((unsigned)((n + 3) / 4), 256, 0, s, p);
    }
    if (e == hipSuccess && p.parts > 1)
        e = launch<scan_sum_ddt>((unsigned)(((int64_t)p.nseq * p.T * p.H + 255) / 256), 256, 0, s, p);
    return e;
}

}  // namespace mil
