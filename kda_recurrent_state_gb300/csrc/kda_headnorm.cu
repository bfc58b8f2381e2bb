// kda_headnorm.cu -- norm of every query and key head with the position rotation in the same pass,
// and its gradients.  For one head x in R^d of a token at position m:
//   r = (mean x^2 + eps)^{-1/2} (RMS), (sum x^2 + eps)^{-1/2} (L2: unit length) or 1 (none)
//   n = r x w            (w: one weight per channel, or 1)
//   y = n with its first `rot` entries turned in pairs (a, b) by the angle of (m, pair):
//       (a cos - b sin, a sin + b cos), pairs (i, i + rot/2) or (2i, 2i + 1).
// Backwards, with g = dy turned back:  dw = sum g r x,   h = g w,
//   dx = r (h - u s <h, u>),  u = r x,   s = 1/d (RMS), 1 (L2);   dx = h (none: x has no part in it)
// (r^3 is never formed: it overflows from norms of 1e-13 down).
//
// Bound by HBM: each head is read once and written once.  A head is held by a power of two of
// lanes, 8 channels each (16 bytes of bf16, 32 of fp32), so its sums are shuffles and the half
// layout's partners one shuffle away (or, where a half is no multiple of 8 channels, in shared
// memory); a lane keeps the angles and weights of its channels while it walks `per_unit` heads of
// a token, whose loads are issued together.  Sizes or alignments that do not allow vectors of 8
// take one warp per head, channel by channel.
//
// Measured (GB300, bf16, d = 128): unit length of 32,768 x 192 heads 0.478 ms, 6.74 TB/s, the copy
// rate; gradients of a weighted norm with 64 turned channels, 32,768 x 40 heads, 0.210 ms, 4.8 TB/s,
// 0.72 of it: the loads of 16 warps an SM (107 registers) and the sums over a head's lanes are waited for, no
// unit is at its limit (issue 58 % busy).
#include "kda_vec.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxHead = 256;
constexpr int kBwdBlocks = 152 * 4;

// 1 / norm, and the factor s of a norm's gradient.
__device__ __forceinline__ float inv_norm(const HeadProblem& p, float ss) {
    if (p.norm == KDA_NORM_NONE) return 1.f;
    return rsqrtf((p.norm == KDA_NORM_RMS ? ss / (float)p.d : ss) + p.eps);
}
__device__ __forceinline__ float grad_share(const HeadProblem& p) {
    return p.norm == KDA_NORM_RMS ? 1.f / (float)p.d : 1.f;
}

// Row of the angle tables for a token, or -1 (not turned): no rotation, or a position outside
// the tables, which raises KDA_STATUS_POSITION_RANGE.
__device__ __forceinline__ int64_t angle_row(const HeadProblem& p, int64_t token) {
    if (p.rot == 0) return -1;
    const int64_t m = p.pos[token];
    if (m < 0 || m >= p.positions) {
        atomicCAS(p.status, 0, (int)KDA_STATUS_POSITION_RANGE);
        return -1;
    }
    return m;
}

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// n floats of a parameter or table; `vec`: from a 16-byte boundary.
template <int n, int m>
__device__ __forceinline__ void ld_floats(const float* src, bool vec, float (&f)[m]) {
    if (vec) {
#pragma unroll
        for (int i = 0; i < n / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(src) + i);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = __ldg(src + i);
    }
}

// The angles of a lane's 8 channels: for halves c[i], s[i] of channel i (s negative in the first
// half, so y = x c + partner s); for neighbours c[j], s[j], j < 4, of its pairs.  The first `live` channels
// are turned; the rest are left as they are, not turned by 0: an infinity or NaN times 0 would spread.
struct Angles {
    float c[8], s[8];
    int live;
};
template <bool kMixed>
__device__ __forceinline__ void load_angles(const HeadProblem& p, int64_t row, int e0, Angles& a) {
#pragma unroll
    for (int i = 0; i < 8; ++i) { a.c[i] = 1.f; a.s[i] = 0.f; }
    a.live = row < 0 ? 0 : p.rot - e0;
    if (a.live <= 0) return;
    const int half = p.rot / 2;
    const float* c = p.cos + row * half;
    const float* s = p.sin + row * half;
    if constexpr (kMixed) {  // the 8 channels may lie in both halves and beyond
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i;
            if (e < p.rot) {
                const bool low = e < half;
                a.c[i] = __ldg(c + (low ? e : e - half));
                const float v = __ldg(s + (low ? e : e - half));
                a.s[i] = low ? -v : v;
            }
        }
    } else if (p.layout == KDA_ROT_HALF) {  // in one half
        const bool low = e0 < half;
        const int k = low ? e0 : e0 - half;
        ld_floats<8>(c + k, p.vec4, a.c);
        ld_floats<8>(s + k, p.vec4, a.s);
#pragma unroll
        for (int i = 0; i < 8; ++i) a.s[i] = low ? -a.s[i] : a.s[i];
    } else if (p.vec4 && e0 + 8 <= p.rot) {
        ld_floats<4>(c + e0 / 2, true, a.c);
        ld_floats<4>(s + e0 / 2, true, a.s);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e0 + 2 * j < p.rot) {
                a.c[j] = __ldg(c + e0 / 2 + j);
                a.s[j] = __ldg(s + e0 / 2 + j);
            }
    }
}
// v turned (sign = 1) or turned back (sign = -1).  `partner`: the lane that holds the other half;
// `ex`: the group's shared memory, 9 floats a lane (an odd distance keeps the banks apart), the ninth 0: the
// partner of a channel that is not turned.
template <bool kMixed>
__device__ __forceinline__ void turn(const HeadProblem& p, const Angles& a, float sign, int partner, int e0, float* ex,
                                     float (&v)[8]) {
    if (p.rot == 0) return;
    if constexpr (kMixed) {
        const int half = p.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) ex[e0 + e0 / 8 + i] = v[i];
        ex[e0 + e0 / 8 + 8] = 0.f;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = e0 + i, o = e < half ? e + half : e - half;
            v[i] = fmaf(v[i], a.c[i], ex[i < a.live ? o + o / 8 : e0 + e0 / 8 + 8] * (sign * a.s[i]));
        }
        __syncwarp();
    } else if (p.layout == KDA_ROT_HALF) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = __shfl_sync(0xffffffffu, v[i], partner);
            const float x = fmaf(v[i], a.c[i], o * (sign * a.s[i]));
            v[i] = a.live > 0 ? x : v[i];  // all of a lane's channels or none
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float x = v[2 * j], y = v[2 * j + 1], s = sign * a.s[j];
            v[2 * j] = 2 * j < a.live ? fmaf(x, a.c[j], -y * s) : x;
            v[2 * j + 1] = 2 * j < a.live ? fmaf(x, s, y * a.c[j]) : y;
        }
    }
}

// What a group of LPH lanes works on: heads [h0, h0 + n) of queries (which = 0) or keys of a token.
struct Unit {
    int64_t token;
    int which, h0, n;
};
__device__ __forceinline__ Unit unit_of(const HeadProblem& p, int64_t u, int64_t total) {
    const int per = p.units[0] + p.units[1];
    Unit r;
    int k;
    if (total < (1ll << 32)) {
        r.token = (uint32_t)u / (uint32_t)per;
        k = (int)((uint32_t)u % (uint32_t)per);
    } else {
        r.token = u / per;
        k = (int)(u % per);
    }
    r.which = k >= p.units[0];
    r.h0 = (r.which ? k - p.units[0] : k) * p.per_unit;
    r.n = min(p.per_unit, p.H[r.which] - r.h0);
    return r;
}
__device__ __forceinline__ int64_t unit_count(const HeadProblem& p) {
    return p.tokens * (p.units[0] + p.units[1]);
}

__device__ __forceinline__ void load_weight(const HeadProblem& p, int which, int e0, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (p.weight[which] && e0 < p.d) ld_floats<8>(p.weight[which] + e0, p.vec4, w);
}

// The partner lane of the half layout, counted in the warp.
template <int LPH>
__device__ __forceinline__ int partner_lane(const HeadProblem& p, int lane) {
    const int in = lane % LPH, q = p.rot / 16;  // lanes of one half
    const int to = in < q ? in + q : in < 2 * q ? in - q : in;
    return lane - in + to;
}

constexpr int kHeads = 4;  // heads of a unit: their loads in flight together

// kMixed: the half layout with halves that are no multiple of 8 channels.
template <typename T, typename To, int LPH, bool kMixed>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(HeadProblem p) {
    __shared__ float s_ex[kMixed ? kThreads * 9 : 1];
    float* const ex = s_ex + (kMixed ? threadIdx.x / LPH * (LPH * 9) : 0);
    const int64_t total = unit_count(p);
    const int64_t u = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / LPH;
    const int lane = threadIdx.x & 31, e0 = (lane % LPH) * 8;
    const bool live = u < total, mine = live && e0 < p.d;
    const Unit un = live ? unit_of(p, u, total) : Unit{0, 0, 0, 0};
    const T* x = static_cast<const T*>(p.x[un.which]) + un.token * p.stride[un.which] + (int64_t)un.h0 * p.d + e0;
    To* y = static_cast<To*>(p.y[un.which]) + (un.token * p.H[un.which] + un.h0) * (int64_t)p.d + e0;
    Raw<T, 8> r[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        memset(&r[k], 0, sizeof(r[k]));
        if (mine && k < un.n) r[k] = ld_raw<T, 8>(x + k * p.d);
    }
    float w[8];
    Angles an;
    load_weight(p, un.which, e0, w);
    load_angles<kMixed>(p, mine ? angle_row(p, un.token) : -1, e0, an);
    const int partner = partner_lane<LPH>(p, lane);
#pragma unroll
    for (int k = 0; k < kHeads; ++k) {
        if (k >= p.per_unit) break;  // the same for the whole grid: every lane takes part in the shuffles
        float v[8];
        widen<T, 8>(r[k], v);
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
        const float inv = inv_norm(p, head_sum<LPH>(ss));
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * inv * w[i];
        turn<kMixed>(p, an, 1.f, partner, e0, ex, v);
        if (mine && k < un.n) st_vec<8>(y + k * p.d, v);
    }
}

// Gradients: the first `q_blocks` blocks take the queries' units, the rest the keys', each with its
// share's stride, so that a thread has one set of weights and of sums of dw.  A block adds its groups'
// sums in order and writes one row of `partial`.  kNorm: there is a norm (a variant without one, because a test at
// every value cost 8 us of 218 at 32,768 x 40 heads of 128 channels).
template <typename T, typename Tg, int LPH, bool kMixed, bool kNorm>
__global__ void __launch_bounds__(kThreads) head_norm_bwd_kernel(HeadProblem p) {
    __shared__ float s_dw[kThreads / LPH][LPH * 8];
    __shared__ float s_ex[kMixed ? kThreads * 9 : 1];
    float* const ex = s_ex + (kMixed ? threadIdx.x / LPH * (LPH * 9) : 0);
    const int lane = threadIdx.x & 31, e0 = (lane % LPH) * 8, group = threadIdx.x / LPH;
    constexpr int groups = kThreads / LPH;
    const int which = (int)blockIdx.x >= p.q_blocks;
    const int block = which ? blockIdx.x - p.q_blocks : blockIdx.x;
    const int blocks = which ? gridDim.x - p.q_blocks : p.q_blocks;
    const int per = p.units[which];
    const int64_t total = p.tokens * per;
    const int partner = partner_lane<LPH>(p, lane);
    const float share = grad_share(p);
    float dw[8], w[8];
    load_weight(p, which, e0, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    for (int64_t base = (int64_t)block * groups; base < total; base += (int64_t)blocks * groups) {
        const int64_t u = base + group;
        const bool live = u < total, mine = live && e0 < p.d;
        int64_t token = 0;
        int h0 = 0;
        if (live) {
            token = total < (1ll << 32) ? (uint32_t)u / (uint32_t)per : u / per;
            h0 = (int)(u - token * per) * p.per_unit;
        }
        const int n = live ? min(p.per_unit, p.H[which] - h0) : 0;
        const T* x = static_cast<const T*>(p.x[which]) + token * p.stride[which] + (int64_t)h0 * p.d + e0;
        const int64_t o = (token * p.H[which] + h0) * (int64_t)p.d + e0;
        const Tg* dy = static_cast<const Tg*>(p.dy[which]) + o;
        Tg* dx = static_cast<Tg*>(p.y[which]) + o;
        Raw<T, 8> rx[kHeads];
        Raw<Tg, 8> rg[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            memset(&rx[k], 0, sizeof(rx[k]));
            memset(&rg[k], 0, sizeof(rg[k]));
            if (mine && k < n) {
                rx[k] = ld_raw<T, 8>(x + k * p.d);
                rg[k] = ld_raw<Tg, 8>(dy + k * p.d);
            }
        }
        Angles an;
        load_angles<kMixed>(p, mine ? angle_row(p, token) : -1, e0, an);
#pragma unroll
        for (int k = 0; k < kHeads; ++k) {
            if (k >= p.per_unit) break;
            float v[8], g[8];
            widen<T, 8>(rx[k], v);
            widen<Tg, 8>(rg[k], g);
            turn<kMixed>(p, an, -1.f, partner, e0, ex, g);
            float ss = 0.f, hx = 0.f, gw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                gw[i] = g[i] * w[i];
                ss = fmaf(v[i], v[i], ss);
                hx = fmaf(gw[i], v[i], hx);
            }
            if constexpr (kNorm) {
                ss = head_sum<LPH>(ss);
                hx = head_sum<LPH>(hx);
                // slots past the unit's heads hold zeros, whose 1 / norm without eps is infinite: they add 0, not NaN, to dw
                const float inv = k < n ? inv_norm(p, ss) : 0.f, along = share * (inv * hx);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float unit = v[i] * inv;
                    dw[i] = fmaf(g[i], unit, dw[i]);
                    v[i] = inv * fmaf(-along, unit, gw[i]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dw[i] = fmaf(g[i], v[i], dw[i]);
                    v[i] = gw[i];
                }
            }
            if (mine && k < n) st_vec<8>(dx + k * p.d, v);
        }
    }
    if (!p.partial) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) s_dw[group][e0 + i] = dw[i];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {  // the other one's half of the row: zeros
        float sum = 0.f;
        if (i / p.d == which)
            for (int g = 0; g < groups; ++g) sum += s_dw[g][i % p.d];
        p.partial[(int64_t)blockIdx.x * 2 * p.d + i] = sum;
    }
}

// ---------------------------------------------------------------- any size: a warp per head
constexpr int kSlots = kMaxHead / 32;

// Channel e of a head in shared memory, turned by the row's angles (sign -1: back).
__device__ __forceinline__ float turned(const HeadProblem& p, const float* v, int e, int64_t row, float sign) {
    if (row < 0 || e >= p.rot) return v[e];
    const int half = p.rot / 2;
    const bool halves = p.layout == KDA_ROT_HALF;
    const int k = halves ? (e < half ? e : e - half) : e / 2;
    const bool first = halves ? e < half : (e & 1) == 0;
    const int other = halves ? (first ? e + half : e - half) : e ^ 1;
    const float c = __ldg(p.cos + row * half + k), s = sign * __ldg(p.sin + row * half + k);
    return fmaf(v[e], c, first ? -v[other] * s : v[other] * s);
}

template <typename T, typename To, bool kBwd>
__global__ void __launch_bounds__(kThreads) head_norm_any_kernel(HeadProblem p) {
    __shared__ float s_v[kThreads / 32][kMaxHead];
    __shared__ float s_dw[kBwd ? 2 : 1][kBwd ? kThreads / 32 : 1][kBwd ? kMaxHead : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* sv = s_v[warp];
    const int64_t heads = p.H[0] + p.H[1], total = p.tokens * heads;
    float dw[2][kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dw[0][i] = dw[1][i] = 0.f;
    for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + warp; u < total;
         u += (int64_t)gridDim.x * (kThreads / 32)) {
        const int64_t token = u / heads;
        int h = (int)(u % heads);
        const int which = h >= p.H[0];
        if (which) h -= p.H[0];
        const T* x = static_cast<const T*>(p.x[which]) + token * p.stride[which] + (int64_t)h * p.d;
        const int64_t o = (token * p.H[which] + h) * (int64_t)p.d;
        const int64_t row = angle_row(p, token);
        float v[kSlots], ss = 0.f;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            const int e = lane + 32 * i;
            v[i] = 0.f;
            if (e < p.d) {
                Raw<T, 1> r = ld_raw<T, 1>(x + e);
                float f[1];
                widen<T, 1>(r, f);
                v[i] = f[0];
            }
            ss = fmaf(v[i], v[i], ss);
        }
        const float inv = inv_norm(p, head_sum<32>(ss));
        __syncwarp();
        if constexpr (!kBwd) {
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int e = lane + 32 * i;
                if (e < p.d) sv[e] = v[i] * inv * (p.weight[which] ? __ldg(p.weight[which] + e) : 1.f);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int e = lane + 32 * i;
                if (e < p.d) {
                    const float f[1] = {turned(p, sv, e, row, 1.f)};
                    st_vec<1>(static_cast<To*>(p.y[which]) + o + e, f);
                }
            }
        } else {
            const To* dy = static_cast<const To*>(p.dy[which]) + o;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int e = lane + 32 * i;
                if (e < p.d) {
                    float f[1];
                    widen<To, 1>(ld_raw<To, 1>(dy + e), f);
                    sv[e] = f[0];
                }
            }
            __syncwarp();
            float g[kSlots], hx = 0.f;
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int e = lane + 32 * i;
                g[i] = 0.f;
                if (e < p.d) {
                    const float t = turned(p, sv, e, row, -1.f);
                    const float n = t * (v[i] * inv);
                    if (which) dw[1][i] += n;
                    else dw[0][i] += n;
                    g[i] = t * (p.weight[which] ? __ldg(p.weight[which] + e) : 1.f);
                }
                hx = fmaf(g[i], v[i], hx);
            }
            const float along = grad_share(p) * (inv * head_sum<32>(hx));
#pragma unroll
            for (int i = 0; i < kSlots; ++i) {
                const int e = lane + 32 * i;
                if (e < p.d) {
                    float f[1] = {inv * fmaf(-along, v[i] * inv, g[i])};
                    // one channel: h and x are parallel, and 1 - x^2 r^2 = eps r^2 takes the place of the difference
                    if (p.d == 1) f[0] = g[i] * inv * (p.eps * inv * inv);
                    if (p.norm == KDA_NORM_NONE) f[0] = g[i];
                    st_vec<1>(static_cast<To*>(p.y[which]) + o + e, f);
                }
            }
        }
    }
    if constexpr (kBwd) {
        if (!p.partial) return;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
            s_dw[0][warp][lane + 32 * i] = dw[0][i];
            s_dw[1][warp][lane + 32 * i] = dw[1][i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.d; i += kThreads) {
            const int which = i / p.d, c = i % p.d;
            float sum = 0.f;
            for (int k = 0; k < kThreads / 32; ++k) sum += s_dw[which][k][c];
            p.partial[((int64_t)blockIdx.x * 2 + which) * p.d + c] = sum;
        }
    }
}

// dw: the blocks' rows of `partial`, added in a fixed order.
__global__ void __launch_bounds__(256) head_dweight_kernel(const float* partial, int blocks, int d, float* dq,
                                                           float* dk) {
    __shared__ float s[8][33];
    const int i = blockIdx.x * 32 + threadIdx.x;
    const int per = (blocks + 7) / 8, lo = per * threadIdx.y, hi = min(lo + per, blocks);
    float sum = 0.f;
    if (i < 2 * d)
#pragma unroll 8
        for (int b = lo; b < hi; ++b) sum += partial[(int64_t)b * 2 * d + i];
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y || i >= 2 * d) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) sum += s[k][threadIdx.x];
    if (i < d) {
        if (dq) dq[i] = sum;
    } else if (dk) {
        dk[i - d] = sum;
    }
}

bool aligned(const void* q, int bytes) { return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0; }

// Vectors of 8: the head a multiple of 8 and every row 16-byte aligned.
bool vector_ok(const HeadProblem& p) {
    if (p.d % 8) return false;
    for (int i = 0; i < 2; ++i)
        if (p.stride[i] % 8 || !aligned(p.x[i], 16) || !aligned(p.y[i], 16) || !aligned(p.dy[i], 16)) return false;
    return true;
}

template <typename T, typename To, bool kBwd, int LPH, bool kMixed>
cudaError_t run_mixed(const HeadProblem& p, int64_t grid, cudaStream_t st) {
    if constexpr (!kBwd) head_norm_kernel<T, To, LPH, kMixed><<<(unsigned)grid, kThreads, 0, st>>>(p);
    else if (p.norm != KDA_NORM_NONE) head_norm_bwd_kernel<T, To, LPH, kMixed, true><<<(unsigned)grid, kThreads, 0, st>>>(p);
    else head_norm_bwd_kernel<T, To, LPH, kMixed, false><<<(unsigned)grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}
template <typename T, typename To, bool kBwd, int LPH>
cudaError_t run_lph(const HeadProblem& p, int64_t grid, cudaStream_t st) {
    return p.layout == KDA_ROT_HALF && p.rot % 16 ? run_mixed<T, To, kBwd, LPH, true>(p, grid, st)
                                                  : run_mixed<T, To, kBwd, LPH, false>(p, grid, st);
}

template <typename T, typename To, bool kBwd>
cudaError_t run(HeadProblem p, cudaStream_t st) {
    const int64_t heads = p.H[0] + p.H[1];
    cudaError_t e;
    int64_t grid = 0;
    if (p.tokens * heads == 0) {
        if (!kBwd) return cudaSuccess;
        e = cudaSuccess;
    } else if (vector_ok(p)) {
        int lph = 1;
        while (lph * 8 < p.d) lph *= 2;
        // Several heads a unit share the angles and keep more bytes in flight, one fills the chip
        // when the heads are few (152 SMs x 16 warps).
        // tables of rot / 2 columns in whole float4, and all from 16-byte boundaries
        p.vec4 = p.rot % 8 == 0 && aligned(p.cos, 16) && aligned(p.sin, 16) && aligned(p.weight[0], 16) &&
                 aligned(p.weight[1], 16);
        p.per_unit = kHeads;
        while (p.per_unit > 1 && p.tokens * heads / p.per_unit * lph < 152 * 16 * 32) p.per_unit >>= 1;
        for (int i = 0; i < 2; ++i) p.units[i] = (p.H[i] + p.per_unit - 1) / p.per_unit;
        const int64_t threads = p.tokens * (p.units[0] + p.units[1]) * lph;
        grid = (threads + kThreads - 1) / kThreads;
        if (kBwd) {  // blocks for the queries and for the keys, by their share of the units
            if (grid > kBwdBlocks) grid = kBwdBlocks;
            const int64_t per = p.units[0] + p.units[1];
            p.q_blocks = (int)((grid * p.units[0] + per - 1) / per);
            if (p.units[0] && p.units[1]) {
                if (grid < 2) grid = 2;
                if (p.q_blocks == grid) --p.q_blocks;
            }
        }
        if (grid > INT32_MAX) return cudaErrorInvalidValue;
        switch (lph) {
            case 1: e = run_lph<T, To, kBwd, 1>(p, grid, st); break;
            case 2: e = run_lph<T, To, kBwd, 2>(p, grid, st); break;
            case 4: e = run_lph<T, To, kBwd, 4>(p, grid, st); break;
            case 8: e = run_lph<T, To, kBwd, 8>(p, grid, st); break;
            case 16: e = run_lph<T, To, kBwd, 16>(p, grid, st); break;
            default: e = run_lph<T, To, kBwd, 32>(p, grid, st); break;
        }
    } else {
        grid = (p.tokens * heads + kThreads / 32 - 1) / (kThreads / 32);
        const int64_t most = kBwd ? kBwdBlocks : 152 * 64;
        if (grid > most) grid = most;
        head_norm_any_kernel<T, To, kBwd><<<(unsigned)grid, kThreads, 0, st>>>(p);
        e = cudaGetLastError();
    }
    if (kBwd && e == cudaSuccess && p.partial) {
        head_dweight_kernel<<<(2 * p.d + 31) / 32, dim3(32, 8), 0, st>>>(p.partial, (int)grid, p.d, p.dweight[0],
                                                                        p.dweight[1]);
        e = cudaGetLastError();
    }
    return e;
}

template <bool kBwd>
cudaError_t dispatch(const HeadProblem& p, int in_dtype, int out_dtype, cudaStream_t st) {
    if (in_dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? run<__nv_bfloat16, __nv_bfloat16, kBwd>(p, st)
                                     : run<__nv_bfloat16, float, kBwd>(p, st);
    return out_dtype == KDA_BF16 ? run<float, __nv_bfloat16, kBwd>(p, st) : run<float, float, kBwd>(p, st);
}

}  // namespace

cudaError_t launch_head_norm(const HeadProblem& p, int in_dtype, int out_dtype, cudaStream_t st) {
    return dispatch<false>(p, in_dtype, out_dtype, st);
}
cudaError_t launch_head_norm_bwd(const HeadProblem& p, int in_dtype, int grad_dtype, cudaStream_t st) {
    return dispatch<true>(p, in_dtype, grad_dtype, st);
}
size_t head_norm_bwd_workspace(int d) { return (size_t)kBwdBlocks * 2 * d * sizeof(float); }

}  // namespace kda
