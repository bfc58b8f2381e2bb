// kda_ssm.cuh -- what the selective scan's forward and backward kernels share: how states and
// channels are spread over a warp, how the token axis is cut into segments, packed fp32 pairs,
// and the loads of 8 channels.
//
// A thread holds 4 (step and gradients) or 8 (scan) neighbouring states of one or two channels, and LN
// neighbouring lanes, a power of two, all of the channels' states.  States past N have A = B = C = 0:
// they stay zero and add zero.
#pragma once

#include "kda_vec.cuh"

namespace kda {
namespace ssm {

// Two fp32 lanes of one register pair; sm_100 multiplies and adds such pairs in one instruction.
struct f2 {
    float x, y;
};
__device__ __forceinline__ unsigned long long bits(f2 a) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ f2 pair(unsigned long long r) {
    f2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(r);
}
__device__ __forceinline__ f2 ex2_2(f2 a) { return f2{ex2(a.x), ex2(a.y)}; }
__device__ __forceinline__ f2 dup(float a) { return f2{a, a}; }

// exp(dt A) with A already times log2 e.  The hardware's 2^x lies on average 0.2 .. 0.9 x 2^-25 below
// the true value for x in [-0.25, 0] (measured, 2^20 points an octave), and a recurrence raises its
// decay to the power of its memory: the exponent is moved up by 0.5 x 2^-25 / ln 2, which takes the
// middle of that bias away where the memory is long (for large |x| it is below the rounding; an exponent of
// 0 still gives exactly 1).  It makes the product dt A a fused operation; times with and without it are the
// same (4 x 8192 x 4096 forward 732 us, 4 x 2048 x 4096 gradients 979 to 983 us, N = 16).
constexpr float kNudge = 2.2e-8f;
// A times log2 e, finite where A is: a step of 0 times an infinite rate would be NaN where exp(0 A) is 1.
// Rates beyond 2.36e38 are taken as they are: any step but 0 (or one below 1e-36) forgets everything.
__device__ __forceinline__ float log2_rate(float A) {
    const float r = kLog2e * A;
    return isinf(r) ? A : r;
}
__device__ __forceinline__ f2 decay2(f2 dt, f2 A) { return ex2_2(fma2(dt, A, dup(kNudge))); }
__device__ __forceinline__ float decay1(float dt, float A) { return ex2(fmaf(dt, A, kNudge)); }

// The token axis in segments of `len` tokens, counted from each sequence's first token.  Segment i
// of sequence s has the slot s * per + i (equal lengths), or cu[s] / len + s + i (packed: distinct,
// with a slot left over here and there).
struct Segments {
    Seqs seqs;
    int64_t len;
    int64_t per;    // segments per sequence, equal lengths
    int64_t slots;  // all of them
};
__host__ __device__ inline Segments make_segments(const Seqs& q, int64_t len) {
    Segments g{q, len, 0, 0};
    if (q.cu) {
        g.slots = q.T_total / len + q.N;
    } else {
        g.per = q.T_uniform > 0 ? (q.T_uniform + len - 1) / len : 1;
        g.slots = g.per * q.N;
    }
    return g;
}
__device__ __forceinline__ int64_t slot_of(const Segments& g, int s, int64_t i) {
    if (!g.seqs.cu) return s * g.per + i;
    return min(max(g.seqs.cu[s], (int64_t)0), g.seqs.T_total) / g.len + s + i;
}
struct Segment {
    int s;             // sequence, -1: an unused slot
    int64_t i, count;  // segment of the sequence, and how many it has
    int64_t a, e;      // the sequence's tokens
    int64_t t0, t1;    // the segment's
};
__device__ __forceinline__ Segment segment_at(const Segments& g, int64_t slot) {
    Segment r;
    if (!g.seqs.cu) {
        r.s = (int)(slot / g.per);
        r.i = slot - r.s * g.per;
    } else {
        int lo = 0, hi = g.seqs.N - 1;  // the last s whose first slot is not above this one
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (slot_of(g, mid, 0) <= slot) lo = mid;
            else hi = mid - 1;
        }
        r.s = lo;
        r.i = slot - slot_of(g, lo, 0);
    }
    seq_range(g.seqs, r.s, r.a, r.e);
    r.count = r.e > r.a ? (r.e - r.a + g.len - 1) / g.len : 1;
    if (r.i < 0 || r.i >= r.count) {
        r.s = -1;
        r.i = 0;
    }
    r.t0 = r.a + r.i * g.len;
    r.t1 = min(r.t0 + g.len, r.e);
    return r;
}

// A group in a thread's own place in shared memory, `stride` bytes between its 16-byte units.
template <typename T>
__device__ __forceinline__ void put_eight(char* dst, int stride, const Raw<T, 8>& r) {
#pragma unroll
    for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i)
        *reinterpret_cast<uint4*>(dst + i * stride) = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
}
// Its elements one by one (past `n`: zeros), in two steps so that other work fits between: loaded into
// registers, and put down.
template <typename T>
struct Pending {
    T v[8];
};
template <typename T>
__device__ __forceinline__ void load_pending(Pending<T>& q, const T* src, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q.v[i] = T(0.f);
        if (i < n) q.v[i] = src[i];
    }
}
template <typename T>
__device__ __forceinline__ void land_pending(char* dst, int stride, const Pending<T>& q) {
    Raw<T, 8> r;
    memset(&r, 0, sizeof(r));
#pragma unroll
    for (int i = 0; i < 8; ++i) set_raw<T, 8>(r, i, q.v[i]);
    put_eight<T>(dst, stride, r);
}
// 8 neighbouring elements of a row into a thread's own place.  kWhole (rows of whole 16-byte units): copied in
// the background, to be waited for; `any` is an address on a 16-byte boundary for the units of which
// nothing is read.  Else at once.
template <bool kWhole, typename T>
__device__ __forceinline__ void copy_eight(char* dst, int stride, const T* src, int n, const void* any) {
    constexpr int kUnits = 8 * (int)sizeof(T) / 16;
    if constexpr (kWhole) {
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            async_copy16(dst + i * stride, n * (int)sizeof(T) > 16 * i ? reinterpret_cast<const char*>(src) + 16 * i : any,
                         n * (int)sizeof(T) > 16 * i);
    } else {
        Pending<T> q;
        load_pending(q, src, n);
        land_pending(dst, stride, q);
    }
}
template <typename T>
__device__ __forceinline__ void take_eight(const char* src, int stride, float (&f)[8]) {
    Raw<T, 8> r;
#pragma unroll
    for (int i = 0; i < 8 * (int)sizeof(T) / 16; ++i) {
        const uint4 v = *reinterpret_cast<const uint4*>(src + i * stride);
        r.w[4 * i] = v.x;
        r.w[4 * i + 1] = v.y;
        r.w[4 * i + 2] = v.z;
        r.w[4 * i + 3] = v.w;
    }
    widen<T, 8>(r, f);
}
// 8 channels to a row of outputs, those past `n` left out; `vec`: rows of whole 16-byte units.
template <typename T>
__device__ __forceinline__ void st_eight(T* p, const float (&f)[8], int n, bool vec) {
    if (vec && n >= 8) {
        st_vec<8>(p, f);
        return;
    }
    if (vec && n >= 4) {  // half a group: fp32 rows of whole 16-byte units
        const float g[4] = {f[0], f[1], f[2], f[3]};
        st_vec<4>(p, g);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < n) {
            const float g[1] = {f[i]};
            st_vec<1>(p + i, g);
        }
}

// softplus and x sigmoid(x) of two values (kda_vec.cuh has the single ones and the derivation).
__device__ __forceinline__ f2 softplus2(f2 x) {
    const f2 e{ex2(-kLog2e * fabsf(x.x)), ex2(-kLog2e * fabsf(x.y))};
    const f2 d = add2(e, dup(2.f)), s = mul2(e, f2{rcp(d.x), rcp(d.y)}), q = mul2(s, s);
    f2 r = fma2(dup(0.14078889156761287f), q, dup(0.13982578878397325f));
    r = fma2(r, q, dup(0.20012297614909472f));
    r = fma2(r, q, dup(0.3333316082070072f));
    r = fma2(r, q, dup(1.000000003840879f));
    return fma2(add2(s, s), r, f2{fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)});
}
__device__ __forceinline__ f2 sigmoid2(f2 x) {
    const f2 e = ex2_2(mul2(x, dup(-kLog2e))), d = add2(e, dup(1.f));
    return f2{rcp(d.x), rcp(d.y)};
}

// Step sizes of 8 channels.  One branch around all of them: a branch per channel would keep their
// chains from overlapping.
__device__ __forceinline__ void step_sizes(float (&raw)[8], bool use_softplus) {
    if (use_softplus)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const f2 r = softplus2(f2{raw[i], raw[i + 1]});
            raw[i] = r.x;
            raw[i + 1] = r.y;
        }
}

// Lanes per state group for N states.
inline int lanes_for(int N) {
    int ln = 1;
    while (4 * ln < N) ln *= 2;
    return ln;
}

inline bool aligned16(const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; }
// Rows and groups of whole 16-byte units (`unit` channels) in every array.
inline bool rows_vector(const SsmProblem& p, int unit) {
    const int64_t per_group = p.D / p.G;
    if (p.D % unit || per_group % unit || p.u_stride % unit || p.delta_stride % unit || (p.z && p.z_stride % unit))
        return false;
    const void* a[] = {p.u, p.delta, p.z, p.out, p.d_out, p.du, p.ddelta, p.dz};
    for (const void* q : a)
        if (!aligned16(q)) return false;
    return true;
}
// The gradients (kda_ssm_bwd.cu).
struct BwdArgs {
    SsmProblem p;
    Segments g, chunks;
    int warps;                          // of a CTA of the last pass: its channels
    int chan_blocks, blocks_per_group;
    bool vec, vec_bc, multi;            // multi: sequences have several segments
    float* ckpt;      // [chunk slots, D, 4 lanes]: the state before each chunk
    float* ckpt_dt;   // [chunk slots, D] sum of dt from the segment's start (several segments)
    float* seg_h;     // [slots, D, N] end states, then start states (0 for a first segment)
    float* seg_g;     // [slots, D, N] start gradients, then end gradients
    float* seg_dt;    // [slots, D]
    float* part;      // [slots, D N + 2 D]: dA, dskip, dbias
    float* part_bc;   // [blocks per group, tokens, G, 2, N]
};
// The passes along the sequences: checkpoints, and with several segments their end states and the
// gradients on their start states (kda_ssm_bwd_scan.cu).
cudaError_t launch_ssm_bwd_scans(const BwdArgs& q, int in_dtype, int grad_dtype, cudaStream_t st);

}  // namespace ssm
}  // namespace kda
