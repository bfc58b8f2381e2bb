// kda_ssm_bwd.cu -- gradients of the selective scan (kda_ssm.cu).  With g_t = dL/dy_t (the gate's
// part taken off: g = d_out z sigmoid(z)), x = dt u and the state's gradient carried from later tokens:
//   dh_t = g_t C_t + a_{t+1} dh_{t+1}
//   dC_t = sum_c g_t h_t       dB_t = sum_c x_t dh_t       (over the channels of the group)
//   du = skip g + dt <dh, B>   d(dt) = u <dh, B> + <dh a h_{t-1}, A>    dA = sum_t dt dh a h_{t-1}
//   ddelta = d(dt) softplus'(.) = d(dt) sigmoid(.)    dz = d_out y sigmoid'(..)    dskip = sum_t g u
//
// The token axis is cut into segments and these into chunks of 4 LN (16 from LN = 4 on) tokens:
//   1. forward over every segment from zero (the first one from the initial state), storing the
//      state at each chunk's start; with more than one segment also the end state and the sum of dt,
//      and, backward in time, the gradient that the segment's own outputs put on its start state;
//   2. (several segments) one walk forward over the end states and one backward over the start
//      gradients: each segment's true start state and end gradient;
//   3. every segment backwards, chunk by chunk: a forward sweep from the chunk's start keeps the
//      state every 4 tokens in shared memory; each group of 4 tokens is then recomputed once more
//      with a and a h_{t-1} in registers and undone in reverse order;
//   4. sums over segments (dA, dskip, dbias) and over channel blocks (dB, dC) in a fixed order.
// The time goes into fp32 work and shuffles, not into the bytes: 3 exponentials and about 20 fp32
// operations per (token, channel, state), which alone take 0.32 ms at 4 x 2048 x 4096, N = 16 (the bytes:
// 0.08 ms).  A thread holds 2 channels x 4 states in (3); the next chunk's rows come by background
// copies while a chunk is worked on.
//
// Measured there: 0.98 ms, of it 0.17 in (1) and 0.80 in (3) (issue 48 %, fp32 38 %, shared memory 55 %
// busy; 7 warps an SM at 229 registers, so latency is exposed, and the phases of a chunk stand between
// barriers).  A group's results are stored after all of its tokens: with a
// store between, the next token's loads waited, and (3) took 0.94 ms.  CTAs of 4 warps, two an SM, cost the
// same (their units do not divide over the SMs), and so did one CTA as two halves with their own
// barriers (0.99 ms); groups of 2 tokens would double the kept states.
#include "kda_ssm.cuh"

namespace kda {
namespace {
using namespace ssm;

constexpr int kGroup = 4;      // tokens undone together
constexpr int kMostWarps = 8;
constexpr float kLn2 = 0.6931471805599453f;

template <int LN> struct Shape {
    static constexpr int kCW = 64 / LN;                // channels of a warp
    static constexpr int kCB = kMostWarps * kCW;       // of a CTA, at most
    static constexpr int kLC = LN <= 4 ? 4 * LN : 16;  // tokens of a chunk
    static constexpr int kN = 4 * LN;
    static constexpr int kNB = kN < 8 ? 8 : kN;        // a row of B or C in shared memory, in states
    static constexpr int kStagers = kLC * kCB / 8;     // threads that stage a group of 8 channels, at most
    static constexpr int kBC = kLC * kNB / 8 * 2;      // groups of 8 states of B and C
    static constexpr int kGroups = kLC / kGroup;
    static constexpr int kKeep = kGroups * 256 * kMostWarps;            // floats: states every 4 tokens
    static constexpr int kRed = kGroups * kMostWarps * kGroup * 2 * kN;  // floats: per-warp dB, dC
    static constexpr bool kAlias = kRed <= kKeep;                       // a group's sums go over its states
    static constexpr int kFloats = 3 * kLC * kCB + 2 * kLC * 2 * kNB + kKeep + (kAlias ? 0 : kRed) +
                                   16 * kStagers + 2 * kCB;
    // raw rows on the way in, two chunks: u, delta, z, d_out, the chunk's start states, B and C
    template <typename T, typename Tg> static constexpr int kSlot =
        kStagers * 8 * (3 * (int)sizeof(T) + (int)sizeof(Tg)) + kMostWarps * 32 * 32 + kBC * 8 * (int)sizeof(T);
    template <typename T, typename Tg> static constexpr int kSmem = kFloats * (int)sizeof(float) + 2 * kSlot<T, Tg>;
};

// ---------------------------------------------------------------- 2. across segments
__global__ void __launch_bounds__(256) ssm_bwd_carry_kernel(BwdArgs q) {
    const SsmProblem& p = q.p;
    const int64_t per = (int64_t)p.D * p.N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * p.seqs.N) return;
    const int s = (int)(i / per);
    const int64_t o = i % per;
    int64_t a, e;
    seq_range(p.seqs, s, a, e);
    const int64_t count = e > a ? (e - a + q.g.len - 1) / q.g.len : 1;
    const float A = log2_rate(p.A[o]);
    const int64_t first = slot_of(q.g, s, 0);
    float* sh = q.seg_h + first * per + o;
    float* sg = q.seg_g + first * per + o;
    const float* dt = q.seg_dt + first * p.D + o / p.N;
    float g = p.d_final ? p.d_final[i] : 0.f;
    if (e <= a) {  // no token: the gradient passes through
        sg[0] = g;
        return;
    }
    float h = sh[0];  // the first segment started from the initial state
    sh[0] = 0.f;
    for (int64_t k0 = 1; k0 < count; k0 += 8) {
        float end[8], d[8];  // eight loads on the way before the first store
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            end[j] = k0 + j < count ? sh[(k0 + j) * per] : 0.f;
            d[j] = k0 + j < count ? dt[(k0 + j) * p.D] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 + j < count) {
                sh[(k0 + j) * per] = h;
                h = fmaf(ex2(A * d[j]), h, end[j]);
            }
    }
    for (int64_t k0 = count - 1; k0 >= 0; k0 -= 8) {
        float start[8], d[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            start[j] = k0 - j >= 0 ? sg[(k0 - j) * per] : 0.f;
            d[j] = k0 - j >= 0 ? dt[(k0 - j) * p.D] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (k0 - j >= 0) {
                sg[(k0 - j) * per] = g;
                g = fmaf(ex2(A * d[j]), g, start[j]);
            }
    }
}

// ---------------------------------------------------------------- 3. backward
// kWhole: rows of channels are whole 16-byte units.
template <typename T, typename Tg, int LN, bool kWhole>
__global__ void __launch_bounds__(32 * kMostWarps, 1) ssm_bwd_kernel(BwdArgs q) {
    using S = Shape<LN>;
    constexpr int LC = S::kLC, NN = S::kN, NB = S::kNB;
    const SsmProblem& p = q.p;
    const int threads = 32 * q.warps, CB = q.warps * S::kCW;
    const int cb = blockIdx.x % q.chan_blocks;
    const int64_t slot = blockIdx.x / q.chan_blocks;
    const Segment seg = segment_at(q.g, slot);

    extern __shared__ __align__(16) float smem[];
    float* s_dt = smem;                  // [LC][CB] dt, then <dh, B>
    float* s_du = s_dt + LC * S::kCB;    // dt u, then <dh a h, A>
    float* s_g = s_du + LC * S::kCB;     // g, then y
    float* s_B = s_g + LC * S::kCB;      // [LC][2 NB] every state twice
    float* s_C = s_B + LC * 2 * NB;
    float* s_keep = s_C + LC * 2 * NB;   // [group][warp][8][32]
    float* s_red = S::kAlias ? s_keep : s_keep + S::kKeep;
    float* s_acc = s_keep + S::kKeep + (S::kAlias ? 0 : S::kRed);  // [16][stagers] dskip, dbias of a stager's channels
    float* s_bias = s_acc + 16 * S::kStagers;                      // [CB]
    float* s_skip = s_bias + S::kCB;
    char* ring = reinterpret_cast<char*>(smem + S::kFloats);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per_group = p.D / p.G, grp = cb / q.blocks_per_group, blk = cb % q.blocks_per_group;
    const int cbase = grp * per_group + blk * CB, cend = min((grp + 1) * per_group, cbase + CB);
    const int ln = lane % LN, cl = warp * S::kCW + (lane / LN) * 2, c0 = cbase + cl;
    const int64_t DN = (int64_t)p.D * p.N;
    float* part = q.part + slot * (DN + 2 * p.D);

    f2 A[4], h[4], dh[4], dA[4], h0[4];
    auto gather = [&](const float* base, f2(&v)[4]) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool st = 4 * ln + n < p.N;
            const int64_t o = (int64_t)c0 * p.N + 4 * ln + n;
            v[n].x = base && st && c0 < cend ? base[o] : 0.f;
            v[n].y = base && st && c0 + 1 < cend ? base[o + p.N] : 0.f;
        }
    };
    auto scatter = [&](float* base, const f2(&v)[4]) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const bool st = 4 * ln + n < p.N;
            const int64_t o = (int64_t)c0 * p.N + 4 * ln + n;
            if (st && c0 < cend) base[o] = v[n].x;
            if (st && c0 + 1 < cend) base[o + p.N] = v[n].y;
        }
    };
    gather(p.A, A);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        A[n] = f2{log2_rate(A[n].x), log2_rate(A[n].y)};
        dA[n] = dup(0.f);
        h0[n] = dup(0.f);
        dh[n] = dup(0.f);
    }
    // a stager's group of 8 channels and its row of a chunk
    const int per_row = CB / 8, srow = tid / per_row, sc = tid % per_row * 8;
    const int sn = srow < LC ? cend - (cbase + sc) : 0;
    float dskip[8], dbias[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dskip[i] = dbias[i] = 0.f;
    for (int i = tid; i < CB; i += threads) {
        s_bias[i] = p.bias && cbase + i < cend ? __ldg(p.bias + cbase + i) : 0.f;
        s_skip[i] = p.skip && cbase + i < cend ? __ldg(p.skip + cbase + i) : 0.f;
    }
    __syncthreads();

    if (seg.s >= 0) {
        if (q.multi) {
            gather(q.seg_g + slot * DN, dh);
            if (seg.i > 0) gather(q.seg_h + slot * DN, h0);
        } else if (p.d_final) {
            gather(p.d_final + seg.s * DN, dh);
        }
        const T* u = static_cast<const T*>(p.u) + cbase + sc;
        const T* dl = static_cast<const T*>(p.delta) + cbase + sc;
        const T* z = p.z ? static_cast<const T*>(p.z) + cbase + sc : nullptr;
        const Tg* dy = static_cast<const Tg*>(p.d_out) + cbase + sc;
        const int64_t chunk0 = slot_of(q.chunks, seg.s, seg.i * (q.g.len / LC));
        const int64_t nchunks = (seg.t1 - seg.t0 + LC - 1) / LC;

        // Every thread copies its own groups in and reads them back: no barrier between.
        constexpr int kUnit = 16 * S::kStagers, kT = 8 * (int)sizeof(T) * S::kStagers;  // bytes
        auto raw = [&](int64_t ch, int g) { return ring + (int)(ch & 1) * S::template kSlot<T, Tg> + g * kT + 16 * tid; };
        auto raw_h = [&](int64_t ch) {
            return ring + (int)(ch & 1) * S::template kSlot<T, Tg> + 3 * kT + 8 * (int)sizeof(Tg) * S::kStagers + 16 * tid;
        };
        auto raw_bc = [&](int64_t ch) { return raw_h(ch) - 16 * tid + kMostWarps * 32 * 32 + 16 * tid; };
        auto fetch = [&](int64_t ch) {
            if (ch >= 0) {
                const int64_t t = seg.t0 + ch * LC;
                if (srow < LC) {
                    const int64_t tt = t + srow;
                    const int n = tt < seg.t1 ? sn : 0;
                    copy_eight<kWhole>(raw(ch, 0), kUnit, u + tt * p.u_stride, n, p.u);
                    copy_eight<kWhole>(raw(ch, 1), kUnit, dl + tt * p.delta_stride, n, p.u);
                    if (z) copy_eight<kWhole>(raw(ch, 2), kUnit, z + tt * p.z_stride, n, p.u);
                    copy_eight<kWhole>(raw(ch, 3), kUnit, dy + tt * p.D, n, p.u);
                }
                const float* ck = q.ckpt + ((chunk0 + ch) * p.D + c0) * NN + 4 * ln;  // rows of 4 LN states, padded
                async_copy16(raw_h(ch), c0 < cend ? ck : q.ckpt, c0 < cend);
                async_copy16(raw_h(ch) + 16 * 32 * kMostWarps, c0 + 1 < cend ? ck + NN : q.ckpt, c0 + 1 < cend);
                for (int e = tid; e < S::kBC; e += threads) {
                    const int which = e / (S::kBC / 2), rr = e % (S::kBC / 2) / (NB / 8), n0 = e % (NB / 8) * 8;
                    const T* src = which ? static_cast<const T*>(p.C) + (t + rr) * p.C_stride
                                         : static_cast<const T*>(p.B) + (t + rr) * p.B_stride;
                    const int n = t + rr < seg.t1 ? p.N - n0 : 0;
                    char* dst = raw_bc(ch) + 16 * (e - tid);
                    if (q.vec_bc) copy_eight<true>(dst, 16 * S::kBC, src + (int64_t)grp * p.N + n0, n, p.B);
                    else copy_eight<false>(dst, 16 * S::kBC, src + (int64_t)grp * p.N + n0, n, p.B);
                }
            }
            async_commit();  // one group a chunk, empty before the first
        };
        fetch(nchunks - 1);

        for (int64_t ch = nchunks - 1; ch >= 0; --ch) {
            const int64_t t = seg.t0 + ch * LC;
            const int tokens = (int)min((int64_t)LC, seg.t1 - t);
            const int n8 = srow < tokens ? sn : 0;
            fetch(ch - 1);
            async_wait<1>();
            // ---- stage (rows past `tokens`: dt = 0, so a = 1 and nothing is added)
            if (srow < LC) {
                float fu[8], fd[8], fg[8], bias[8];
                take_eight<T>(raw(ch, 0), kUnit, fu);
                take_eight<T>(raw(ch, 1), kUnit, fd);
                take_eight<Tg>(raw(ch, 3), kUnit, fg);
                widen<float, 8>(ld_raw<float, 8>(s_bias + sc), bias);
#pragma unroll
                for (int i = 0; i < 8; ++i) fd[i] += bias[i];
                step_sizes(fd, p.softplus);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    fd[i] = n8 > 0 ? fd[i] : 0.f;
                    fu[i] *= fd[i];
                }
                if (z) {
                    float fz[8];
                    take_eight<T>(raw(ch, 2), kUnit, fz);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const f2 zz{fz[i], fz[i + 1]}, r = mul2(zz, sigmoid2(zz));
                        fg[i] *= r.x;
                        fg[i + 1] *= r.y;
                    }
                }
                st_vec<8>(s_dt + srow * CB + sc, fd);
                st_vec<8>(s_du + srow * CB + sc, fu);
                st_vec<8>(s_g + srow * CB + sc, fg);
            }
            for (int e = tid; e < S::kBC; e += threads) {
                float f[8];
                take_eight<T>(raw_bc(ch) + 16 * (e - tid), 16 * S::kBC, f);
                float* o = (e < S::kBC / 2 ? s_B : s_C) + e % (S::kBC / 2) * 16;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4*>(o + 4 * i) = make_float4(f[2 * i], f[2 * i], f[2 * i + 1], f[2 * i + 1]);
            }
            {  // the state before the chunk
                const float4 a = *reinterpret_cast<const float4*>(raw_h(ch));
                const float4 b = *reinterpret_cast<const float4*>(raw_h(ch) + 16 * 32 * kMostWarps);
                h[0] = f2{a.x, b.x};
                h[1] = f2{a.y, b.y};
                h[2] = f2{a.z, b.z};
                h[3] = f2{a.w, b.w};
            }
            if (q.multi && seg.i > 0) {
                const float* cd = q.ckpt_dt + (chunk0 + ch) * p.D;
                const f2 d{c0 < cend ? cd[c0] : 0.f, c0 + 1 < cend ? cd[c0 + 1] : 0.f};
#pragma unroll
                for (int n = 0; n < 4; ++n) h[n] = fma2(ex2_2(mul2(A[n], d)), h0[n], h[n]);
            }
            __syncthreads();

            auto pairs = [&](const float* row, f2(&v)[4]) {  // 4 states, each twice
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float4 w = *reinterpret_cast<const float4*>(row + 8 * ln + 4 * n);
                    v[2 * n] = f2{w.x, w.y};
                    v[2 * n + 1] = f2{w.z, w.w};
                }
            };
            auto two = [&](const float* s, int i) {
                const float2 v = *reinterpret_cast<const float2*>(s + i * CB + cl);
                return f2{v.x, v.y};
            };
            const int groups = (tokens + kGroup - 1) / kGroup;
            f2 dAc[4];  // the chunk's part of dA: two levels of sums keep the rounding of long ones small
#pragma unroll
            for (int n = 0; n < 4; ++n) dAc[n] = dup(0.f);
            // ---- forward sweep: the state before every group
            for (int j = 0; j < groups; ++j) {
                float* keep = s_keep + (j * kMostWarps + warp) * 256 + lane;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    keep[64 * n] = h[n].x;
                    keep[64 * n + 32] = h[n].y;
                }
                if (j + 1 == groups) break;
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const int k = j * kGroup + i;
                    const f2 d = two(s_dt, k), x = two(s_du, k);
                    f2 b[4];
                    pairs(s_B + k * 2 * NB, b);
#pragma unroll
                    for (int n = 0; n < 4; ++n) h[n] = fma2(decay2(d, A[n]), h[n], mul2(x, b[n]));
                }
            }
            // ---- groups backwards
            for (int j = groups - 1; j >= 0; --j) {
                const float* keep = s_keep + (j * kMostWarps + warp) * 256 + lane;
                f2 hh[4], a[kGroup][4], ah[kGroup][4];
#pragma unroll
                for (int n = 0; n < 4; ++n) hh[n] = f2{keep[64 * n], keep[64 * n + 32]};
                __syncwarp();  // the sums of dB and dC go over these states
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const int k = j * kGroup + i;  // rows past `tokens` hold dt = 0: a = 1, nothing added
                    const f2 d = two(s_dt, k), x = two(s_du, k);
                    f2 b[4];
                    pairs(s_B + k * 2 * NB, b);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        a[i][n] = decay2(d, A[n]);
                        ah[i][n] = mul2(a[i][n], hh[n]);
                        hh[n] = fma2(x, b[n], ah[i][n]);
                    }
                }
                float* red = S::kAlias ? s_keep + (j * kMostWarps + warp) * 256 : s_red + (j * kMostWarps + warp) * kGroup * 2 * NN;
                // What the group's tokens leave is stored after all of them: a store between would hold back
                // the next token's loads.
                constexpr int kLast = LN >= 16 ? 4 : LN == 8 ? 2 : 1;  // values of dB, dC that a lane ends with
                float rv[kGroup][kLast], r0[kGroup], r1[kGroup], r2[kGroup];
                f2 p0[LN == 1 ? kGroup : 1], p1[LN == 1 ? kGroup : 1], p2[LN == 1 ? kGroup : 1];
                int idx = 0;
                bool writes = true;
#pragma unroll
                for (int i = kGroup - 1; i >= 0; --i) {
                    const int k = j * kGroup + i;
                    const f2 d = two(s_dt, k), x = two(s_du, k), g = two(s_g, k);
                    f2 b[4], c[4], y = dup(0.f), inner = dup(0.f), gA = dup(0.f);
                    pairs(s_B + k * 2 * NB, b);
                    pairs(s_C + k * 2 * NB, c);
                    float v[8];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const f2 H = fma2(x, b[n], ah[i][n]);
                        dh[n] = fma2(g, c[n], dh[n]);
                        y = fma2(c[n], H, y);
                        const f2 dc = mul2(g, H), db = mul2(x, dh[n]);
                        v[n] = db.x + db.y;
                        v[4 + n] = dc.x + dc.y;
                        inner = fma2(dh[n], b[n], inner);
                        const f2 w = mul2(dh[n], ah[i][n]);
                        gA = fma2(w, A[n], gA);
                        dAc[n] = fma2(w, d, dAc[n]);
                        dh[n] = mul2(a[i][n], dh[n]);
                    }
                    // over the warp's channels: halves of the live values exchanged while there are several
                    idx = 0;
                    writes = true;
                    int live = 8;
#pragma unroll
                    for (int o = 16; o >= LN; o >>= 1) {
                        if (live > 1) {
                            live >>= 1;
                            const bool up = lane & o;
#pragma unroll
                            for (int m = 0; m < 4; ++m)
                                if (m < live) {
                                    const float send = up ? v[m] : v[m + live];
                                    v[m] = (up ? v[m + live] : v[m]) + __shfl_xor_sync(0xffffffffu, send, o);
                                }
                            if (up) idx += live;
                        } else {
                            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
                            writes = writes && !(lane & o);
                        }
                    }
#pragma unroll
                    for (int m = 0; m < kLast; ++m) rv[i][m] = v[m];
                    // over the lanes of a channel
                    if constexpr (LN > 1) {
                        const bool odd = lane & 1;
                        r0[i] = (odd ? inner.y : inner.x) + __shfl_xor_sync(0xffffffffu, odd ? inner.x : inner.y, 1);
                        r1[i] = (odd ? gA.y : gA.x) + __shfl_xor_sync(0xffffffffu, odd ? gA.x : gA.y, 1);
                        r2[i] = (odd ? y.y : y.x) + __shfl_xor_sync(0xffffffffu, odd ? y.x : y.y, 1);
#pragma unroll
                        for (int o = 2; o < LN; o <<= 1) {
                            r0[i] += __shfl_xor_sync(0xffffffffu, r0[i], o);
                            r1[i] += __shfl_xor_sync(0xffffffffu, r1[i], o);
                            r2[i] += __shfl_xor_sync(0xffffffffu, r2[i], o);
                        }
                    } else {
                        p0[i] = inner;
                        p1[i] = gA;
                        p2[i] = y;
                    }
                }
                __syncwarp();  // every lane has read the group's rows
#pragma unroll
                for (int i = 0; i < kGroup; ++i) {
                    const int k = j * kGroup + i;
#pragma unroll
                    for (int m = 0; m < kLast; ++m) {
                        const int id = idx + m;  // 0..3: dB of state 4 ln + id, 4..7: dC
                        if (writes) red[i * 2 * NN + (id >> 2) * NN + 4 * ln + (id & 3)] = rv[i][m];
                    }
                    if constexpr (LN > 1) {
                        if (ln < 2) {
                            s_dt[k * CB + cl + (lane & 1)] = r0[i];
                            s_du[k * CB + cl + (lane & 1)] = r1[i];
                            s_g[k * CB + cl + (lane & 1)] = r2[i];
                        }
                    } else {
                        *reinterpret_cast<float2*>(s_dt + k * CB + cl) = make_float2(p0[i].x, p0[i].y);
                        *reinterpret_cast<float2*>(s_du + k * CB + cl) = make_float2(p1[i].x, p1[i].y);
                        *reinterpret_cast<float2*>(s_g + k * CB + cl) = make_float2(p2[i].x, p2[i].y);
                    }
                }
            }
#pragma unroll
            for (int n = 0; n < 4; ++n) dA[n] = add2(dA[n], dAc[n]);
            __syncthreads();
            // ---- finish the chunk's rows (their places in shared memory are the stager's own)
            if (n8 > 0) {
                float fu[8], fd[8], fg[8], in[8], ga[8], sk[8], bias[8];
                take_eight<T>(raw(ch, 0), kUnit, fu);
                take_eight<T>(raw(ch, 1), kUnit, fd);
                take_eight<Tg>(raw(ch, 3), kUnit, fg);
                widen<float, 8>(ld_raw<float, 8>(s_dt + srow * CB + sc), in);
                widen<float, 8>(ld_raw<float, 8>(s_du + srow * CB + sc), ga);
                widen<float, 8>(ld_raw<float, 8>(s_skip + sc), sk);
                widen<float, 8>(ld_raw<float, 8>(s_bias + sc), bias);
                const int64_t o = (t + srow) * p.D + cbase + sc;
                if (z) {
                    float fz[8], yy[8];
                    take_eight<T>(raw(ch, 2), kUnit, fz);
                    widen<float, 8>(ld_raw<float, 8>(s_g + srow * CB + sc), yy);
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const f2 zz{fz[i], fz[i + 1]}, sg = sigmoid2(zz), gg{fg[i], fg[i + 1]};
                        const f2 full = fma2(f2{sk[i], sk[i + 1]}, f2{fu[i], fu[i + 1]}, f2{yy[i], yy[i + 1]});
                        const f2 gs = mul2(gg, sg), gz = mul2(gs, zz);
                        // z' silu: sg (1 + z (1 - sg))
                        const f2 slope = fma2(zz, fma2(sg, dup(-1.f), dup(1.f)), dup(1.f));
                        const f2 dz = mul2(mul2(gs, full), slope);
                        yy[i] = dz.x;
                        yy[i + 1] = dz.y;
                        fg[i] = gz.x;
                        fg[i + 1] = gz.y;
                    }
                    st_eight(static_cast<Tg*>(p.dz) + o, yy, n8, kWhole);
                }
                float dt[8], slope[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dt[i] = fd[i] + bias[i];
                    slope[i] = 1.f;
                }
                if (p.softplus)
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const f2 raw2{dt[i], dt[i + 1]}, s2 = sigmoid2(raw2), d2 = softplus2(raw2);
                        slope[i] = s2.x;
                        slope[i + 1] = s2.y;
                        dt[i] = d2.x;
                        dt[i + 1] = d2.y;
                    }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    fd[i] = fmaf(fu[i], in[i], ga[i] * kLn2) * slope[i];
                    dskip[i] = fmaf(fg[i], fu[i], dskip[i]);
                    dbias[i] += fd[i];
                    fu[i] = fmaf(dt[i], in[i], sk[i] * fg[i]);
                }
                st_eight(static_cast<Tg*>(p.du) + o, fu, n8, kWhole);
                st_eight(static_cast<Tg*>(p.ddelta) + o, fd, n8, kWhole);
            }
            for (int i = tid; i < tokens * 2 * NN / 4; i += threads) {  // 4 states of dB or dC over the warps
                const int row = i / (NN / 2), v = i % (NN / 2) * 4, n = v % NN;
                const float* r = (S::kAlias ? s_keep + (row / kGroup) * kMostWarps * 256
                                            : s_red + (row / kGroup) * kMostWarps * kGroup * 2 * NN) +
                                 (row % kGroup) * 2 * NN + v;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kMostWarps; ++w)
                    if (w < q.warps) {
                        const float4 x = *reinterpret_cast<const float4*>(r + w * (S::kAlias ? 256 : kGroup * 2 * NN));
                        sum.x += x.x;
                        sum.y += x.y;
                        sum.z += x.z;
                        sum.w += x.w;
                    }
                float* o = q.part_bc + ((((int64_t)blk * p.seqs.T_total + t + row) * p.G + grp) * 2 + v / NN) * p.N + n;
                const float f[4] = {sum.x, sum.y, sum.z, sum.w};
                if (p.N % 4 == 0) {
                    if (n < p.N) st_vec<4>(o, f);
                } else {
#pragma unroll
                    for (int m = 0; m < 4; ++m)
                        if (n + m < p.N) o[m] = f[m];
                }
            }
        }
        if (seg.i == 0 && p.d_init) scatter(p.d_init + seg.s * DN, dh);
    }
    scatter(part, dA);
    // dskip and dbias over the rows of the stagers
    if (srow < LC)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            s_acc[i * S::kStagers + tid] = dskip[i];
            s_acc[(8 + i) * S::kStagers + tid] = dbias[i];
        }
    __syncthreads();
    for (int i = tid; i < 2 * CB; i += threads) {
        const int c = i % CB, which = i / CB;
        if (cbase + c >= cend) continue;
        float sum = 0.f;
        for (int r = 0; r < LC; ++r) sum += s_acc[(which * 8 + c % 8) * S::kStagers + r * per_row + c / 8];
        part[DN + which * p.D + cbase + c] = sum;
    }
}

// ---------------------------------------------------------------- 4. sums in a fixed order
// dA, dskip and dbias over the slots.
__global__ void __launch_bounds__(256) ssm_bwd_sum_kernel(BwdArgs q) {
    __shared__ float s[8][33];
    const SsmProblem& p = q.p;
    const int64_t DN = (int64_t)p.D * p.N, M = DN + 2 * p.D;
    const int64_t i = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const int64_t per = (q.g.slots + 7) / 8, lo = per * threadIdx.y, hi = min(lo + per, q.g.slots);
    float sum = 0.f;
    if (i < M)
#pragma unroll 8
        for (int64_t k = lo; k < hi; ++k) sum += q.part[k * M + i];
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y || i >= M) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) sum += s[k][threadIdx.x];
    if (i < DN) p.dA[i] = sum;
    else if (i < DN + p.D) {
        if (p.dskip) p.dskip[i - DN] = sum;
    } else if (p.dbias) {
        p.dbias[i - DN - p.D] = sum;
    }
}

// dB and dC over the channel blocks of a group.  kSplit: 32 neighbouring values a block, eight runs of
// channel blocks side by side (for few values, each of up to 256 partial sums); else a value a thread.
template <bool kSplit>
__global__ void __launch_bounds__(256) ssm_bwd_bc_kernel(BwdArgs q) {
    __shared__ float s[8][33];
    const SsmProblem& p = q.p;
    const int64_t M = p.seqs.T_total * p.G * 2 * p.N;
    const int x = threadIdx.x % 32, y = threadIdx.x / 32;
    const int64_t i = kSplit ? (int64_t)blockIdx.x * 32 + x : (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per = kSplit ? (q.blocks_per_group + 7) / 8 : q.blocks_per_group;
    const int lo = kSplit ? per * y : 0, hi = min(lo + per, q.blocks_per_group);
    float sum = 0.f;
    if (i < M)
#pragma unroll 4
        for (int b = lo; b < hi; ++b) sum += q.part_bc[b * M + i];
    if constexpr (kSplit) {
        s[y][x] = sum;
        __syncthreads();
        if (y) return;
#pragma unroll
        for (int k = 1; k < 8; ++k) sum += s[k][x];
    }
    if (i >= M) return;
    const int64_t row = i / (2 * p.N);
    const int v = (int)(i % (2 * p.N));
    if (v < p.N) p.dB[row * p.N + v] = sum;
    else p.dC[row * p.N + v - p.N] = sum;
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int chunk_len(int N) {
    const int ln = lanes_for(N);
    return ln <= 4 ? 4 * ln : 16;
}

// Warps of a CTA, and tokens of a segment: whole sequences where (sequence, channel block) pairs fill
// the chip, else one segment an SM.
void cut(const SsmProblem& p, int& warps, int64_t& len) {
    const int cw = 64 / lanes_for(p.N), per_group = p.D / p.G, step = cw < 8 ? 8 / cw : 1;
    auto blocks = [&](int w) { return (int64_t)p.G * ((per_group + w * cw - 1) / (w * cw)); };
    int most = kMostWarps;
    while (most > step && (most - step) * cw >= per_group) most -= step;
    warps = most;
    if (!p.seqs.cu && p.seqs.N * blocks(most) >= 96) {
        int64_t cost = INT64_MAX;  // as for the prompt: the number of warps that fills the last wave best
        for (int w = most; w > most / 2; w -= step) {
            const int64_t c = (p.seqs.N * blocks(w) + 151) / 152 * w;
            if (c < cost) {
                cost = c;
                warps = w;
            }
        }
        len = (p.seqs.T_uniform + 63) / 64 * 64;
    } else {
        len = (p.seqs.T_total * blocks(most) + 151) / 152;
        if (p.seqs.T_total <= 128) len = p.seqs.T_total;  // not worth a walk over segments
        len = (len + 63) / 64 * 64;
    }
    if (len < 64) len = 64;
}

// The workspace's layout; with `base` null only its size.
size_t layout(BwdArgs& q, char* base) {
    const SsmProblem& p = q.p;
    int64_t len;
    cut(p, q.warps, len);
    const int cb = q.warps * (64 / lanes_for(p.N));
    q.blocks_per_group = (p.D / p.G + cb - 1) / cb;
    q.chan_blocks = p.G * q.blocks_per_group;
    q.g = make_segments(p.seqs, len);
    q.chunks = make_segments(p.seqs, chunk_len(p.N));
    q.multi = p.seqs.cu ? len < p.seqs.T_total : q.g.per > 1;
    size_t at = 0;
    auto take = [&](float*& ptr, int64_t floats) {
        ptr = base ? reinterpret_cast<float*>(base + at) : nullptr;
        at += align256((size_t)floats * sizeof(float));
    };
    const int64_t DN = (int64_t)p.D * p.N;
    take(q.ckpt, q.chunks.slots * p.D * 4 * lanes_for(p.N));
    take(q.part, q.g.slots * (DN + 2 * p.D));
    take(q.part_bc, q.blocks_per_group * p.seqs.T_total * p.G * 2 * p.N);
    if (q.multi) {
        take(q.ckpt_dt, q.chunks.slots * p.D);
        take(q.seg_h, q.g.slots * DN);
        take(q.seg_g, q.g.slots * DN);
        take(q.seg_dt, q.g.slots * p.D);
    }
    return at;
}

template <typename T, typename Tg, int LN, bool kWhole>
cudaError_t run_ln(const BwdArgs& q, cudaStream_t st) {
    using S = Shape<LN>;
    const SsmProblem& p = q.p;
    const int64_t grid = q.g.slots * q.chan_blocks, DN = (int64_t)p.D * p.N;
    const int64_t carry = (DN * p.seqs.N + 255) / 256, sums = (DN + 2 * p.D + 31) / 32;
    if (grid > INT32_MAX || carry > INT32_MAX || sums > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = S::template kSmem<T, Tg>;
    static_assert(smem <= 227 * 1024, "a CTA's shared memory");
    auto* bwd = ssm_bwd_kernel<T, Tg, LN, kWhole>;
    const cudaError_t e = cudaFuncSetAttribute(bwd, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (q.multi) ssm_bwd_carry_kernel<<<(unsigned)carry, 256, 0, st>>>(q);
    bwd<<<(unsigned)grid, 32 * q.warps, smem, st>>>(q);
    ssm_bwd_sum_kernel<<<(unsigned)sums, dim3(32, 8), 0, st>>>(q);
    if (p.seqs.T_total > 0) {
        const int64_t values = p.seqs.T_total * p.G * 2 * p.N;
        if ((values + 255) / 256 > INT32_MAX) return cudaErrorInvalidValue;
        if (values < 1 << 18) ssm_bwd_bc_kernel<true><<<(unsigned)((values + 31) / 32), 256, 0, st>>>(q);
        else ssm_bwd_bc_kernel<false><<<(unsigned)((values + 255) / 256), 256, 0, st>>>(q);
    }
    return cudaGetLastError();
}

template <typename T, typename Tg, int LN>
cudaError_t run_whole(const BwdArgs& q, cudaStream_t st) {
    return q.vec ? run_ln<T, Tg, LN, true>(q, st) : run_ln<T, Tg, LN, false>(q, st);
}

template <typename T, typename Tg>
cudaError_t run(const BwdArgs& q, cudaStream_t st) {
    switch (lanes_for(q.p.N)) {
        case 1: return run_whole<T, Tg, 1>(q, st);
        case 2: return run_whole<T, Tg, 2>(q, st);
        case 4: return run_whole<T, Tg, 4>(q, st);
        case 8: return run_whole<T, Tg, 8>(q, st);
        default: return run_whole<T, Tg, 16>(q, st);
    }
}

}  // namespace

size_t ssm_bwd_workspace(int64_t seqs, int64_t T_total, int D, int N, int G, bool packed) {
    BwdArgs q{};
    q.p.D = D;
    q.p.N = N;
    q.p.G = G;
    q.p.seqs = Seqs{packed ? reinterpret_cast<const int64_t*>(8) : nullptr,  // only looked at for null
                    packed || seqs == 0 ? 0 : T_total / seqs, T_total, (int)seqs};
    return layout(q, nullptr);
}

cudaError_t launch_ssm_bwd(const SsmProblem& p, int in_dtype, int grad_dtype, void* workspace, cudaStream_t st) {
    BwdArgs q{};
    q.p = p;
    layout(q, static_cast<char*>(workspace));
    const int unit = in_dtype == KDA_F32 && grad_dtype == KDA_F32 ? 4 : 8;
    q.vec = rows_vector(p, unit);
    q.vec_bc = p.N % unit == 0 && p.B_stride % unit == 0 && p.C_stride % unit == 0 && aligned16(p.B) && aligned16(p.C);
    const cudaError_t e = launch_ssm_bwd_scans(q, in_dtype, grad_dtype, st);
    if (e != cudaSuccess) return e;
    if (in_dtype == KDA_BF16)
        return grad_dtype == KDA_BF16 ? run<__nv_bfloat16, __nv_bfloat16>(q, st) : run<__nv_bfloat16, float>(q, st);
    return grad_dtype == KDA_BF16 ? run<float, __nv_bfloat16>(q, st) : run<float, float>(q, st);
}

}  // namespace kda
