// kda_ssm_scan.cuh -- the scan over tokens of the selective state space operator, for prompts and for
// the passes of the gradients that run along a sequence.
//
// A CTA owns up to 256 / LN channels and walks a segment of a sequence, tile of tokens by tile.  Its
// helper warps stage a tile (dt and dt u in fp32) and finish an earlier one (skip, gate, one rounding)
// while its scan warps, with 2 channels x 8 states a thread in registers, run the tile between: the
// scan's chains of fp32 and exponential work are not interrupted by loads, softplus or the gate.
//
// What bounds it: per (token, 32 channels x 16 states) 32 fp32 operations on register pairs, each occupying
// the operand ports for 2 (product) to 3 (fused, three different operands) cycles, about 80 cycles of a
// scheduler, and beside them 16 exponentials, 64 cycles of their unit.  4 x 8192 x 4096 takes 170 cycles
// and 104 instructions (0.73 ms on the 128 SMs that its 128-channel blocks fill): issue 56 %, fp32 pipes
// 50 % with the helpers' work, exponentials 39 %.  No unit is at its limit; one scan warp and one helper warp
// a scheduler leave the latency of their chains exposed.
//
// Tried and slower: 1 channel x 8 states a thread on 148 SMs (0.77 ms: twice the loads of B and C);
// 8 helper warps (0.82: they take issue slots from the scan); the next token's decays computed ahead
// by hand (0.75); sums of scalars in place of pairs (+18 %); 2 CTAs an SM at 128 registers (0.77 here,
// 8 % faster from 300 CTAs on); raw tiles prefetched into registers (1.09: they must land before the
// barrier); 4 tokens in flight (0.76) against 8.
#pragma once

#include <type_traits>

#include "kda_ssm.cuh"

namespace kda {
namespace ssm {

constexpr int kMostScan = 4, kHelpWarps = 4;  // warps of a CTA; the scan warps of a launch: ScanArgs::scan_warps
constexpr int kHelp = 32 * kHelpWarps;
constexpr int kUnroll = 8;  // tokens of a scan thread in flight

// What a scan is run for:
//   kOutputs    the prompt: outputs and final states, segments from their true start states
//   kEnds       the first pass of a split prompt: end states from zero and sums of dt
//   kKeep       the gradients' first pass: the state before every chunk (and, when the token axis is
//               split, what kEnds leaves); a sequence's first segment starts from its initial state
//   kBack       the same backwards in time for the state's gradient: dh = a (dh + g C), from zero;
//               leaves the gradient that a segment's own outputs put on its start state
enum class Scan { kOutputs, kEnds, kKeep, kBack };

struct ScanArgs {
    SsmProblem p;
    Segments g;
    int scan_warps;
    int chan_blocks;        // per slot
    int blocks_per_group;
    bool vec, vec_state, vec_bc;
    float* seg_state;       // [slots, D, N]: end states from zero, then start states; or nullptr
    float* seg_dt;          // [slots, D]: sums of dt
    float* seg_grad;        // [slots, D, N] (kBack)
    Segments chunks;        // kKeep: chunks of chunks.len tokens, a power of two; segments are whole ones
    float* ckpt;            // [chunk slots, D, ckpt_n]
    float* ckpt_dt;         // [chunk slots, D], or nullptr (token axis not split)
    int ckpt_n;             // N rounded up to 4 lanes' states
};

// A scan thread holds the states 8 ln .. 8 ln + 7 of 2 channels, LN lanes the N <= 8 LN states.
template <int LN> struct ScanShape {
    static constexpr int kCW = 64 / LN;                // channels of a warp
    static constexpr int kCB = kMostScan * kCW;        // of a CTA, at most
    static constexpr int kTT = LN <= 4 ? 8 * LN : 32;  // tokens of a tile
    static constexpr int kN = 8 * LN;
    static constexpr int kVec = kTT * kCB / 8 / kHelp;              // groups of 8 channels a helper stages, at most
    static constexpr int kBC = (2 * kTT * LN + kHelp - 1) / kHelp;  // groups of 8 states of B and C
    static constexpr int kStage = kTT * (2 * kCB + 2 * kN);         // floats of a staged tile
    static constexpr int kFloats = 2 * (kStage + kTT * kCB) + 2 * kCB;
    // raw tiles on the way in: per helper thread kVec groups of u, delta and z and kBC of B and C
    static constexpr int kRaw = 3 * kVec + kBC;
    static constexpr int kRing = 4;
    template <typename T> static constexpr int kSmem = kFloats * (int)sizeof(float) +
                                                       kRing * kRaw * kHelp * 8 * (int)sizeof(T);
};

// The wider type of a launch's raw tiles: kBack reads d_out in the place of u.
template <typename T, typename To, Scan kMode>
using ScanWide = std::conditional_t<kMode == Scan::kBack && (sizeof(To) > sizeof(T)), To, T>;

// (dt, dt u) of two channels lie in 16 bytes, chunk c of a row at chunk swz(c): the helpers' 64-byte
// writes and the scan's reads both touch all banks.
__device__ __forceinline__ int swz(int chunk) { return chunk ^ ((chunk >> 3) & 3); }

// In step i the scan warps work on tile i while the helper warps stage tile i + 1 and finish tile
// i - 1; one barrier a step.  Loads into registers would have to land before the barrier, so the raw
// tiles come by background copies, two steps ahead.
// kWhole: rows of channels are whole 16-byte units.
// To: the outputs' type; for kBack that of d_out.
template <typename T, typename To, int LN, Scan kMode, bool kWhole>
__global__ void __launch_bounds__(32 * (kMostScan + kHelpWarps), 1) scan_kernel(ScanArgs q) {
    using S = ScanShape<LN>;
    constexpr int TT = S::kTT, NN = S::kN;
    constexpr bool kMain = kMode == Scan::kOutputs, kBackward = kMode == Scan::kBack;
    const SsmProblem& p = q.p;
    const int CB = q.scan_warps * S::kCW;
    const int cb = blockIdx.x % q.chan_blocks;
    const int64_t slot = blockIdx.x / q.chan_blocks;
    const Segment seg = segment_at(q.g, slot);
    if (seg.s < 0) return;
    if (kMode == Scan::kEnds && seg.i + 1 == seg.count) return;  // nothing starts from the last segment's end
    if (kBackward && seg.i == 0) return;                         // nor ends at the first one's start

    extern __shared__ __align__(16) float smem[];
    // stage b: (dt, dt u) [TT][CB], B [TT][NN], C [TT][NN]; y of tile b [TT][CB]; bias, skip [CB]
    auto stage = [&](int64_t b) { return smem + (b & 1) * S::kStage; };
    auto ybuf = [&](int64_t b) { return smem + 2 * S::kStage + (b & 1) * TT * S::kCB; };

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per_group = p.D / p.G, grp = cb / q.blocks_per_group;
    const int cbase = grp * per_group + (cb % q.blocks_per_group) * CB;
    const int cend = min((grp + 1) * per_group, cbase + CB);
    const int64_t tiles = (seg.t1 - seg.t0 + TT - 1) / TT;
    auto tile_at = [&](int64_t i) { return seg.t0 + (kBackward ? tiles - 1 - i : i) * TT; };  // first token of step i's tile

    if (warp < q.scan_warps) {
        const int ln = lane % LN, cl = warp * S::kCW + lane / LN * 2, c0 = cbase + cl;
        f2 A[2][4], h[2][4];
        float sum_dt[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                float av[2], hv[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const int st = 8 * ln + 2 * n + m;
                    const bool in = c0 + k < cend && st < p.N;
                    const int64_t o = (int64_t)(c0 + k) * p.N + st;
                    av[m] = in ? log2_rate(__ldg(p.A + o)) : 0.f;
                    hv[m] = 0.f;
                    if (kMain && in && q.seg_state && seg.count > 1) hv[m] = q.seg_state[slot * p.D * p.N + o];
                    else if ((kMain || (kMode == Scan::kKeep && seg.i == 0)) && in && p.init)
                        hv[m] = p.init[(int64_t)seg.s * p.D * p.N + o];
                }
                A[k][n] = f2{av[0], av[1]};
                h[k][n] = f2{hv[0], hv[1]};
            }
        const int at = 4 * swz(cl / 2), row = 2 * CB;
        const int64_t chunk0 = kMode == Scan::kKeep ? slot_of(q.chunks, seg.s, seg.i * (q.g.len / q.chunks.len)) : 0;
        const int chunk_shift = 31 - __clz((int)q.chunks.len);
        auto keep = [&](int64_t t) {  // the state before token t
            const int64_t chunk = chunk0 + ((int)(t - seg.t0) >> chunk_shift);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (c0 + k < cend) {
                    float* o = q.ckpt + (chunk * p.D + c0 + k) * q.ckpt_n + 8 * ln;
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const float v[4] = {h[k][2 * n].x, h[k][2 * n].y, h[k][2 * n + 1].x, h[k][2 * n + 1].y};
                        if (8 * ln + 4 * n < q.ckpt_n) st_vec<4>(o + 4 * n, v);
                    }
                    if (q.ckpt_dt && ln == 0) q.ckpt_dt[chunk * p.D + c0 + k] = sum_dt[k];
                }
        };
        __syncthreads();
        for (int64_t i = 0; i <= tiles; ++i) {
            if (i < tiles) {
                const float* s_dx = stage(i) + at;
                const float* s_B = stage(i) + TT * 2 * S::kCB + 8 * ln;
                const float* s_C = s_B + TT * NN;
                float* s_y = ybuf(i) + cl;
                const int64_t t = tile_at(i);
                const int tokens = (int)min((int64_t)TT, seg.t1 - t);
                // `count` tokens, their outputs stored after all of them: a store between would hold
                // back the next token's loads, and with them everything that could overlap
                auto group = [&](int j0, auto count) {
                    constexpr int U = decltype(count)::value;
                    float r0[U], r1[U];
#pragma unroll
                    for (int jj = 0; jj < U; ++jj) {
                        const int j = kBackward ? tokens - 1 - j0 - jj : j0 + jj;
                        // tested only where a chunk can start: a branch at every token would keep the tokens apart
                        if (kMode == Scan::kKeep && (LN == 1 ? jj % 4 == 0 : jj == 0) &&
                            ((int)(t - seg.t0) + j & (int)(q.chunks.len - 1)) == 0)
                            keep(t + j);
                        const float4 dx = *reinterpret_cast<const float4*>(s_dx + j * row);
                        const f2 d[2] = {dup(dx.x), dup(dx.z)}, x[2] = {dup(dx.y), dup(dx.w)};
                        f2 b[4], c[4], y[2];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float4 v = *reinterpret_cast<const float4*>(s_B + j * NN + 4 * n);
                            b[2 * n] = f2{v.x, v.y};
                            b[2 * n + 1] = f2{v.z, v.w};
                            if (kMain) {
                                const float4 w = *reinterpret_cast<const float4*>(s_C + j * NN + 4 * n);
                                c[2 * n] = f2{w.x, w.y};
                                c[2 * n + 1] = f2{w.z, w.w};
                            }
                        }
                        if (!kMain && !kBackward) {
                            sum_dt[0] += dx.x;
                            sum_dt[1] += dx.z;
                        }
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                if (kBackward) {  // x is the output's gradient and b is C
                                    h[k][n] = mul2(decay2(d[k], A[k][n]), fma2(x[k], b[n], h[k][n]));
                                    continue;
                                }
                                h[k][n] = fma2(decay2(d[k], A[k][n]), h[k][n], mul2(x[k], b[n]));
                                if (kMain) y[k] = n == 0 ? mul2(c[n], h[k][n]) : fma2(c[n], h[k][n], y[k]);
                            }
                        if (kMain) {
                            r0[jj] = y[0].x + y[0].y;
                            r1[jj] = y[1].x + y[1].y;
                            if constexpr (LN > 1) {  // even lanes end with the first channel, odd ones with the second
                                const bool odd = lane & 1;
                                r0[jj] = (odd ? r1[jj] : r0[jj]) + __shfl_xor_sync(0xffffffffu, odd ? r0[jj] : r1[jj], 1);
#pragma unroll
                                for (int o = 2; o < LN; o <<= 1) r0[jj] += __shfl_xor_sync(0xffffffffu, r0[jj], o);
                            }
                        }
                    }
                    if constexpr (kMain) {
#pragma unroll
                        for (int jj = 0; jj < U; ++jj) {
                            float* o = s_y + (j0 + jj) * CB;
                            if constexpr (LN == 1) *reinterpret_cast<float2*>(o) = make_float2(r0[jj], r1[jj]);
                            else if (ln < 2) o[lane & 1] = r0[jj];
                        }
                    }
                };
                int j = 0;
                for (; j + kUnroll <= tokens; j += kUnroll) group(j, std::integral_constant<int, kUnroll>{});
                for (; j < tokens; ++j) group(j, std::integral_constant<int, 1>{});
            }
            __syncthreads();
        }
        float* end = kMain ? (seg.i + 1 == seg.count && p.final_state ? p.final_state + (int64_t)seg.s * p.D * p.N : nullptr)
                     : kBackward                   ? q.seg_grad + slot * p.D * p.N
                     : q.seg_state                 ? q.seg_state + slot * p.D * p.N
                                                   : nullptr;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (c0 + k >= cend) continue;
            if (end) {
                float* o = end + (int64_t)(c0 + k) * p.N + 8 * ln;
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const float v[4] = {h[k][2 * n].x, h[k][2 * n].y, h[k][2 * n + 1].x, h[k][2 * n + 1].y};
                    if (q.vec_state) {
                        if (8 * ln + 4 * n < p.N) st_vec<4>(o + 4 * n, v);
                    } else {
#pragma unroll
                        for (int m = 0; m < 4; ++m)
                            if (8 * ln + 4 * n + m < p.N) o[4 * n + m] = v[m];
                    }
                }
            }
            if (!kMain && !kBackward && q.seg_state && ln == 0) q.seg_dt[slot * p.D + c0 + k] = sum_dt[k];
        }
        return;
    }

    // ---- helper warps
    const int tid = threadIdx.x - 32 * q.scan_warps;
    const int per_row = CB / 8, groups = TT * per_row;
    int row[S::kVec], sc[S::kVec];  // a thread's groups of 8 channels; row TT: none
#pragma unroll
    for (int k = 0; k < S::kVec; ++k) {
        const int e = tid + k * kHelp;
        row[k] = e < groups ? e / per_row : TT;
        sc[k] = e < groups ? e % per_row * 8 : 0;
    }
    float* const s_bias = smem + 2 * (S::kStage + TT * S::kCB);
    float* const s_skip = s_bias + S::kCB;
    for (int i = tid; i < CB; i += kHelp) {
        s_bias[i] = p.bias && cbase + i < cend ? __ldg(p.bias + cbase + i) : 0.f;
        s_skip[i] = kMain && p.skip && cbase + i < cend ? __ldg(p.skip + cbase + i) : 0.f;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kHelp) : "memory");  // the helpers alone
    const T* u = static_cast<const T*>(p.u) + cbase;
    const T* dl = static_cast<const T*>(p.delta) + cbase;
    const T* z = p.z ? static_cast<const T*>(p.z) + cbase : nullptr;
    const To* dy = static_cast<const To*>(p.d_out) + cbase;  // kBack
    // Every helper thread copies its own groups in and reads them back: no barrier between.
    constexpr int kUnit = 16 * kHelp;                        // bytes between a group's 16-byte units
    constexpr int kGroupBytes = 8 * (int)sizeof(ScanWide<T, To, kMode>) * kHelp;  // between groups
    char* const ring = reinterpret_cast<char*>(smem + S::kFloats) + 16 * tid;
    auto raw = [&](int64_t i, int g) { return ring + ((int)(i & 3) * S::kRaw + g) * kGroupBytes; };
    // What cannot be copied in the background is loaded into registers at a step's start and put down at
    // its end: registers would have to land before the barrier anyhow, and the step's work lies between.
    Pending<T> pend[kWhole ? 1 : 3 * S::kVec], pend_bc[S::kBC];
    Pending<To> pend_g[kWhole || !kBackward ? 1 : S::kVec];
    auto fetch = [&](int64_t i) {  // tile i on its way
        if (i < tiles) {
            const int64_t t = tile_at(i);
#pragma unroll
            for (int k = 0; k < S::kVec; ++k) {
                const int64_t tt = t + row[k];
                const int n = row[k] < TT && tt < seg.t1 ? cend - cbase - sc[k] : 0;
                const bool gate = (kMain || kBackward) && z;
                if constexpr (kWhole) {
                    if constexpr (kBackward) copy_eight<true>(raw(i, 3 * k), kUnit, dy + tt * p.D + sc[k], n, p.u);
                    else copy_eight<true>(raw(i, 3 * k), kUnit, u + tt * p.u_stride + sc[k], n, p.u);
                    copy_eight<true>(raw(i, 3 * k + 1), kUnit, dl + tt * p.delta_stride + sc[k], n, p.u);
                    if (gate) copy_eight<true>(raw(i, 3 * k + 2), kUnit, z + tt * p.z_stride + sc[k], n, p.u);
                } else {
                    if constexpr (kBackward) load_pending(pend_g[k], dy + tt * p.D + sc[k], n);
                    else load_pending(pend[3 * k], u + tt * p.u_stride + sc[k], n);
                    load_pending(pend[3 * k + 1], dl + tt * p.delta_stride + sc[k], n);
                    if (gate) load_pending(pend[3 * k + 2], z + tt * p.z_stride + sc[k], n);
                }
            }
#pragma unroll
            for (int k = 0; k < S::kBC; ++k) {
                const int e = tid + k * kHelp, which = e / (TT * LN), rr = e % (TT * LN) / LN, n0 = e % LN * 8;
                if (which > (kMain ? 1 : 0)) continue;
                const T* src = (which || kBackward ? static_cast<const T*>(p.C) + (t + rr) * p.C_stride
                                                   : static_cast<const T*>(p.B) + (t + rr) * p.B_stride) +
                               (int64_t)grp * p.N + n0;
                const int n = t + rr < seg.t1 ? p.N - n0 : 0;
                if (q.vec_bc) copy_eight<true>(raw(i, 3 * S::kVec + k), kUnit, src, n, p.B);
                else load_pending(pend_bc[k], src, n);
            }
        }
        async_commit();  // one group a tile, empty past the end
    };
    auto land = [&](int64_t i) {
        if (i >= tiles) return;
        if constexpr (!kWhole) {
#pragma unroll
            for (int k = 0; k < S::kVec; ++k) {
                if constexpr (kBackward) land_pending(raw(i, 3 * k), kUnit, pend_g[k]);
                else land_pending(raw(i, 3 * k), kUnit, pend[3 * k]);
                land_pending(raw(i, 3 * k + 1), kUnit, pend[3 * k + 1]);
                if ((kMain || kBackward) && z) land_pending(raw(i, 3 * k + 2), kUnit, pend[3 * k + 2]);
            }
        }
        if (!q.vec_bc) {
#pragma unroll
            for (int k = 0; k < S::kBC; ++k)
                if ((tid + k * kHelp) / (TT * LN) <= (kMain ? 1 : 0)) land_pending(raw(i, 3 * S::kVec + k), kUnit, pend_bc[k]);
        }
    };
    auto put = [&](int64_t i) {  // tile i for the scan
        float* s = stage(i);
#pragma unroll
        for (int k = 0; k < S::kVec; ++k) {
            if (row[k] == TT) continue;
            float fu[8], fd[8], bias[8];
            if constexpr (kBackward) {  // g in the place of dt u
                take_eight<To>(raw(i, 3 * k), kUnit, fu);
                if (z) {
                    float fz[8];
                    take_eight<T>(raw(i, 3 * k + 2), kUnit, fz);
#pragma unroll
                    for (int m = 0; m < 8; m += 2) {
                        const f2 zz{fz[m], fz[m + 1]}, r = mul2(zz, sigmoid2(zz));
                        fu[m] *= r.x;
                        fu[m + 1] *= r.y;
                    }
                }
            } else {
                take_eight<T>(raw(i, 3 * k), kUnit, fu);
            }
            take_eight<T>(raw(i, 3 * k + 1), kUnit, fd);
            widen<float, 8>(ld_raw<float, 8>(s_bias + sc[k]), bias);
#pragma unroll
            for (int m = 0; m < 8; ++m) fd[m] += bias[m];
            step_sizes(fd, p.softplus);
            if (!kBackward)
#pragma unroll
                for (int m = 0; m < 8; ++m) fu[m] *= fd[m];
#pragma unroll
            for (int m = 0; m < 4; ++m)  // rows past the segment's end are not scanned
                *reinterpret_cast<float4*>(s + row[k] * 2 * CB + 4 * swz(sc[k] / 2 + m)) =
                    make_float4(fd[2 * m], fu[2 * m], fd[2 * m + 1], fu[2 * m + 1]);
        }
#pragma unroll
        for (int k = 0; k < S::kBC; ++k) {
            const int e = tid + k * kHelp;
            if (e >= (kMain ? 2 : 1) * TT * LN) continue;
            float f[8];
            take_eight<T>(raw(i, 3 * S::kVec + k), kUnit, f);
            st_vec<8>(s + TT * 2 * S::kCB + e * 8, f);  // B of all tokens, then C: [which][row][n]
        }
    };
    fetch(0);
    land(0);
    fetch(1);
    land(1);
    async_wait<1>();
    if (tiles > 0) put(0);
    __syncthreads();
    for (int64_t i = 0; i <= tiles; ++i) {
        fetch(i + 2);  // over tile i - 2, which is finished
        async_wait<1>();
        if (i + 1 < tiles) put(i + 1);
        if constexpr (kMain) {
            const int64_t t = seg.t0 + (i - 1) * TT;
            const float* s = ybuf(i - 1);
#pragma unroll
            for (int k = 0; k < S::kVec; ++k) {
                const int sn = cend - cbase - sc[k];
                if (i == 0 || row[k] == TT || t + row[k] >= seg.t1 || sn <= 0) continue;
                float fu[8], o[8], skip[8];
                take_eight<T>(raw(i - 1, 3 * k), kUnit, fu);
                widen<float, 8>(ld_raw<float, 8>(s + row[k] * CB + sc[k]), o);
                widen<float, 8>(ld_raw<float, 8>(s_skip + sc[k]), skip);
#pragma unroll
                for (int m = 0; m < 8; ++m) o[m] = fmaf(skip[m], fu[m], o[m]);
                if (z) {
                    float fz[8];
                    take_eight<T>(raw(i - 1, 3 * k + 2), kUnit, fz);
#pragma unroll
                    for (int m = 0; m < 8; m += 2) {
                        const f2 zz{fz[m], fz[m + 1]}, r = mul2(f2{o[m], o[m + 1]}, mul2(zz, sigmoid2(zz)));
                        o[m] = r.x;
                        o[m + 1] = r.y;
                    }
                }
                st_eight(static_cast<To*>(p.out) + (t + row[k]) * p.D + cbase + sc[k], o, sn, kWhole);
            }
        }
        land(i + 2);
        __syncthreads();
    }
}

// Lanes per channel of the scan.
inline int scan_lanes(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }

// How a prompt is cut: scan warps of a CTA (its channels), and tokens of a segment.
struct ScanPlan {
    int scan_warps;
    int64_t len;
};
inline ScanPlan scan_plan(int64_t seqs, int64_t T_total, int64_t T_uniform, int D, int G, int N, bool packed) {
    const int cw = 64 / scan_lanes(N), per_group = D / G;  // cw: whole groups of 8 channels
    auto blocks = [&](int w) { return (int64_t)G * ((per_group + w * cw - 1) / (w * cw)); };
    int most = kMostScan;
    while (most > 1 && (most - 1) * cw >= per_group) --most;
    if (!packed && seqs * blocks(most) >= 96) {
        // Whole sequences fill the chip: of 3 or 4 scan warps the number whose CTAs, one an SM, fill
        // their last wave best (fewer warps would leave an SM's pipes idle).
        int best = most;
        int64_t cost = INT64_MAX;
        for (int w = most; w > most / 2; --w) {
            const int64_t c = (seqs * blocks(w) + 151) / 152 * w;
            if (c < cost) {
                cost = c;
                best = w;
            }
        }
        return {best, T_uniform > 0 ? T_uniform : 1};
    }
    // One segment an SM; three where packed sequences of different lengths leave segments of different
    // lengths (16384 x 1024 in one sequence: 154 us with 1, 171 with 3; ragged fp32: 177 with 1, 165 with 3).
    const int64_t want = packed ? 456 : 152;
    int64_t len = (T_total * blocks(most) + want - 1) / want;
    len = (len + 31) / 32 * 32;
    return {most, len < 128 ? 128 : len};
}

// Launches one mode over all segments; q.scan_warps, q.g and q.vec.. set, q.chan_blocks set here.
template <typename T, typename To, int LN, Scan kMode, bool kWhole>
cudaError_t launch_scan_ln(ScanArgs q, cudaStream_t st) {
    using S = ScanShape<LN>;
    const SsmProblem& p = q.p;
    const int cb = q.scan_warps * S::kCW;
    q.blocks_per_group = (p.D / p.G + cb - 1) / cb;
    q.chan_blocks = p.G * q.blocks_per_group;
    const int64_t grid = q.g.slots * q.chan_blocks;
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = S::template kSmem<ScanWide<T, To, kMode>>;
    auto* fn = scan_kernel<T, To, LN, kMode, kWhole>;
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    fn<<<(unsigned)grid, 32 * (q.scan_warps + kHelpWarps), smem, st>>>(q);
    return cudaGetLastError();
}
template <typename T, typename To, Scan kMode>
cudaError_t launch_scan(const ScanArgs& q, cudaStream_t st) {
    const bool whole = q.vec;
    switch (scan_lanes(q.p.N)) {
        case 1: return whole ? launch_scan_ln<T, To, 1, kMode, true>(q, st) : launch_scan_ln<T, To, 1, kMode, false>(q, st);
        case 2: return whole ? launch_scan_ln<T, To, 2, kMode, true>(q, st) : launch_scan_ln<T, To, 2, kMode, false>(q, st);
        case 4: return whole ? launch_scan_ln<T, To, 4, kMode, true>(q, st) : launch_scan_ln<T, To, 4, kMode, false>(q, st);
        default: return whole ? launch_scan_ln<T, To, 8, kMode, true>(q, st) : launch_scan_ln<T, To, 8, kMode, false>(q, st);
    }
}

}  // namespace ssm
}  // namespace kda
