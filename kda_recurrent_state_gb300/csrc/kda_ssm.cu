// kda_ssm.cu -- the selective state space scan: per channel c a state h in R^N, with B and C shared
// by the channels of a group,
//   dt = softplus(delta_t + bias) (or delta_t + bias)      a = exp(dt A)
//   h_t = a h_{t-1} + dt u_t B_t        y_t = <C_t, h_t> + skip u_t        out_t = y_t z_t sigmoid(z_t).
//
// Work per (token, channel): N exponentials and 4 N fp32 operations against 6 to 8 bytes of bf16: for
// N = 16 the fp32 units need 1.7 times the time of the bytes, and the scan takes 2.6 times theirs
// (kda_ssm_scan.cuh says why).
//
// Prompt: the scan of kda_ssm_scan.cuh, a CTA per (sequence, block of channels).
// With too few (sequence, channel) pairs to fill the chip the token axis is cut into segments:
// their end states from zero (first pass), one walk over the segments, then the scan proper
// from each segment's true start.
//
// Single tokens: bound by the state's bytes, read once and written once.
//
// Measured (GB300, bf16 activations, N = 16): prompt 4 x 8192 x 4096 0.73 ms (bytes alone: 0.16 ms), one
// sequence of 16,384 x 1024 0.15 ms (0.06 first pass, 0.01 walk, 0.08 outputs); step of 256 x 8192
// 0.057 ms, 5.1 TB/s, 0.76 of the copy rate.
#include "kda_ssm_scan.cuh"

namespace kda {
namespace {
using namespace ssm;

// Start states of the segments from their end states from zero: one thread per (sequence, channel, state).
__global__ void __launch_bounds__(256) scan_carry_kernel(ScanArgs q) {
    const SsmProblem& p = q.p;
    const int64_t per = (int64_t)p.D * p.N;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per * p.seqs.N) return;
    const int s = (int)(i / per);
    const int64_t o = i % per;
    const int c = (int)(o / p.N);
    int64_t a, e;
    seq_range(p.seqs, s, a, e);
    const int64_t count = e > a ? (e - a + q.g.len - 1) / q.g.len : 1;
    if (count == 1) return;
    const float A = log2_rate(p.A[o]);
    float h = p.init ? p.init[i] : 0.f;
    const int64_t first = slot_of(q.g, s, 0);
    float* st = q.seg_state + first * per + o;
    const float* dt = q.seg_dt + first * p.D + c;
    for (int64_t k0 = 0; k0 < count; k0 += 8) {
        float end[8], d[8];  // eight loads on the way before the first store
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool more = k0 + j + 1 < count;  // the last segment's end is not in the table
            end[j] = more ? st[(k0 + j) * per] : 0.f;
            d[j] = more ? dt[(k0 + j) * p.D] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 + j < count) st[(k0 + j) * per] = h;
            h = fmaf(ex2(A * d[j]), h, end[j]);
        }
    }
}

// One token per session.  A thread holds 4 states of a channel of SESS sessions: A is read once for
// them, and all their loads are on the way before the first is used (sessions past the last read
// the last one's and store nothing).  What a (session, channel) has once -- its step, input, gate and
// output -- belongs to one of the channel's LN lanes: it loads it, hands the step on by shuffles, and
// ends the exchange of the partial outputs with the sum.
template <typename T, typename To, int LN, int SESS>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs q, unsigned gx) {
    const SsmProblem& p = q.p;
    const int ln = threadIdx.x % LN, n0 = 4 * ln;
    const int64_t c64 = ((int64_t)(blockIdx.x % gx) * 256 + threadIdx.x) / LN;
    const bool in_c = c64 < p.D, some = n0 < p.N;
    const int c = in_c ? (int)c64 : p.D - 1;
    const int b0 = blockIdx.x / gx * SESS, last = p.seqs.N - 1;
    const int grp = c / (p.D / p.G);
    Raw<float, 4> rh[SESS];
    Raw<T, 4> rB[SESS], rC[SESS];
    constexpr int OWNERS = LN < SESS ? LN : SESS, OWN = SESS / OWNERS;
    const int lane = threadIdx.x & 31, first = ln % OWNERS * OWN;  // own sessions: first .. first + OWN - 1
    Raw<T, 1> ru[OWN], rd[OWN], rz[OWN];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        const int64_t b = min(b0 + first + k, last);
        ru[k] = ld_raw<T, 1>(static_cast<const T*>(p.u) + b * p.u_stride + c);
        rd[k] = ld_raw<T, 1>(static_cast<const T*>(p.delta) + b * p.delta_stride + c);
        if (p.z) rz[k] = ld_raw<T, 1>(static_cast<const T*>(p.z) + b * p.z_stride + c);
    }
#pragma unroll
    for (int k = 0; k < SESS; ++k) {
        const int64_t b = min(b0 + k, last);
        const float* st = p.final_state + (b * p.D + c) * p.N + n0;
        const T* Bp = static_cast<const T*>(p.B) + b * p.B_stride + (int64_t)grp * p.N + n0;
        const T* Cp = static_cast<const T*>(p.C) + b * p.C_stride + (int64_t)grp * p.N + n0;
        memset(&rh[k], 0, sizeof(rh[k]));
        memset(&rB[k], 0, sizeof(rB[k]));
        memset(&rC[k], 0, sizeof(rC[k]));
        if (q.vec_state) {
            if (some) rh[k] = ld_raw<float, 4>(st);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n0 + n < p.N) set_raw<float, 4>(rh[k], n, st[n]);
        }
        if (q.vec_bc) {
            if (some) rB[k] = ld_raw<T, 4>(Bp);
            if (some) rC[k] = ld_raw<T, 4>(Cp);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n0 + n < p.N) {
                    set_raw<T, 4>(rB[k], n, Bp[n]);
                    set_raw<T, 4>(rC[k], n, Cp[n]);
                }
        }
    }
    float A[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) A[n] = n0 + n < p.N ? log2_rate(__ldg(p.A + (int64_t)c * p.N + n0 + n)) : 0.f;
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f, skip = p.skip ? __ldg(p.skip + c) : 0.f;
    float dt[OWN], u[OWN], y[SESS];
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        float f[1];
        widen<T, 1>(rd[k], f);
        dt[k] = f[0] + bias;
        widen<T, 1>(ru[k], f);
        u[k] = f[0];
    }
    if (p.softplus)
#pragma unroll
        for (int k = 0; k < OWN; ++k) dt[k] = softplus(dt[k]);
#pragma unroll
    for (int k = 0; k < SESS; ++k) {
        float h[4], B[4], C[4];
        widen<float, 4>(rh[k], h);
        widen<T, 4>(rB[k], B);
        widen<T, 4>(rC[k], C);
        const int from = lane - ln + k / OWN;  // the owner
        const float d = OWNERS > 1 ? __shfl_sync(0xffffffffu, dt[k % OWN], from) : dt[k % OWN];
        const float x = d * (OWNERS > 1 ? __shfl_sync(0xffffffffu, u[k % OWN], from) : u[k % OWN]);
        y[k] = 0.f;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            h[n] = fmaf(decay1(d, A[n]), h[n], x * B[n]);
            y[k] = fmaf(C[n], h[n], y[k]);
        }
        if (!in_c || b0 + k > last) continue;
        float* st = p.final_state + ((int64_t)(b0 + k) * p.D + c) * p.N + n0;
        if (q.vec_state) {
            if (some) st_vec<4>(st, h);
        } else {
#pragma unroll
            for (int n = 0; n < 4; ++n)
                if (n0 + n < p.N) st[n] = h[n];
        }
    }
    // the owners' sums: halves of the sessions exchanged, then whole sums over the lanes beyond the owners
#pragma unroll
    for (int o = OWNERS / 2, live = SESS / 2; o >= 1; o >>= 1, live >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int m = 0; m < SESS / 2; ++m)
            if (m < live) {
                const float send = up ? y[m] : y[m + live];
                y[m] = (up ? y[m + live] : y[m]) + __shfl_xor_sync(0xffffffffu, send, o);
            }
    }
#pragma unroll
    for (int o = OWNERS; o < LN; o <<= 1)
#pragma unroll
        for (int k = 0; k < OWN; ++k) y[k] += __shfl_xor_sync(0xffffffffu, y[k], o);
    if (!in_c || ln >= OWNERS) return;
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
        float o[1] = {fmaf(skip, u[k], y[k])}, f[1];
        if (p.z) {
            widen<T, 1>(rz[k], f);
            o[0] *= f[0] * sigmoid(f[0]);
        }
        if (b0 + first + k <= last) st_vec<1>(static_cast<To*>(p.out) + (int64_t)(b0 + first + k) * p.D + c, o);
    }
}

template <typename T, typename To>
cudaError_t fwd(const ScanArgs& q, cudaStream_t st) {
    if (q.seg_state) {
        const int64_t carry = ((int64_t)q.p.seqs.N * q.p.D * q.p.N + 255) / 256;
        if (carry > INT32_MAX) return cudaErrorInvalidValue;
        const cudaError_t e = launch_scan<T, T, Scan::kEnds>(q, st);
        if (e != cudaSuccess) return e;
        scan_carry_kernel<<<(unsigned)carry, 256, 0, st>>>(q);
    }
    return launch_scan<T, To, Scan::kOutputs>(q, st);
}

template <typename T, typename To, int LN>
cudaError_t step_ln(const ScanArgs& q, cudaStream_t st) {
    const SsmProblem& p = q.p;
    const int64_t gx = ((int64_t)p.D * LN + 255) / 256;
    // 4 sessions a thread, or 1 while 4 would leave SMs idle.
    const int sess = gx * ((p.seqs.N + 3) / 4) < 152 * 4 ? 1 : 4;
    const int64_t gy = (p.seqs.N + sess - 1) / sess;
    if (gx * gy > INT32_MAX) return cudaErrorInvalidValue;
    if (sess == 4) scan_step_kernel<T, To, LN, 4><<<(unsigned)(gx * gy), 256, 0, st>>>(q, (unsigned)gx);
    else scan_step_kernel<T, To, LN, 1><<<(unsigned)(gx * gy), 256, 0, st>>>(q, (unsigned)gx);
    return cudaGetLastError();
}

template <typename T, typename To>
cudaError_t run(const ScanArgs& q, bool step, cudaStream_t st) {
    if (step) switch (lanes_for(q.p.N)) {
            case 1: return step_ln<T, To, 1>(q, st);
            case 2: return step_ln<T, To, 2>(q, st);
            case 4: return step_ln<T, To, 4>(q, st);
            case 8: return step_ln<T, To, 8>(q, st);
            default: return step_ln<T, To, 16>(q, st);
        }
    return fwd<T, To>(q, st);
}

cudaError_t dispatch(const ScanArgs& q, bool step, int in_dtype, int out_dtype, cudaStream_t st) {
    if (in_dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? run<__nv_bfloat16, __nv_bfloat16>(q, step, st)
                                     : run<__nv_bfloat16, float>(q, step, st);
    return out_dtype == KDA_BF16 ? run<float, __nv_bfloat16>(q, step, st) : run<float, float>(q, step, st);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t ssm_fwd_workspace(int64_t seqs, int64_t T_total, int D, int N, int G, bool packed) {
    const int64_t T = packed || seqs == 0 ? 0 : T_total / seqs;
    const int64_t len = scan_plan(seqs, T_total, T, D, G, N, packed).len;
    if (packed ? len >= T_total : len >= T) return 0;
    const Seqs s{packed ? reinterpret_cast<const int64_t*>(1) : nullptr, T, T_total, (int)seqs};  // cu: only looked at for null
    const size_t slots = (size_t)make_segments(s, len).slots;
    return align256(slots * D * N * sizeof(float)) + align256(slots * D * sizeof(float));
}

cudaError_t launch_ssm_fwd(const SsmProblem& p, int in_dtype, int out_dtype, void* workspace, cudaStream_t st) {
    ScanArgs q{};
    q.p = p;
    const ScanPlan how = scan_plan(p.seqs.N, p.seqs.T_total, p.seqs.T_uniform, p.D, p.G, p.N, p.seqs.cu != nullptr);
    q.scan_warps = how.scan_warps;
    q.g = make_segments(p.seqs, how.len);
    const int unit = in_dtype == KDA_F32 && out_dtype == KDA_F32 ? 4 : 8;  // elements of a 16-byte unit, in and out
    q.vec = rows_vector(p, unit);
    q.vec_state = p.N % 4 == 0 && aligned16(p.final_state) && aligned16(workspace);
    q.vec_bc = p.N % unit == 0 && p.B_stride % unit == 0 && p.C_stride % unit == 0 && aligned16(p.B) && aligned16(p.C);
    if (ssm_fwd_workspace(p.seqs.N, p.seqs.T_total, p.D, p.N, p.G, p.seqs.cu != nullptr)) {
        q.seg_state = static_cast<float*>(workspace);
        q.seg_dt = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                            align256((size_t)q.g.slots * p.D * p.N * sizeof(float)));
    }
    return dispatch(q, false, in_dtype, out_dtype, st);
}

cudaError_t launch_ssm_step(const SsmProblem& p, int in_dtype, int out_dtype, cudaStream_t st) {
    ScanArgs q{};
    q.p = p;
    q.vec_state = p.N % 4 == 0 && aligned16(p.final_state);
    const uintptr_t four = in_dtype == KDA_BF16 ? 8 : 16;
    q.vec_bc = p.N % 4 == 0 && p.B_stride % 4 == 0 && p.C_stride % 4 == 0 &&
               reinterpret_cast<uintptr_t>(p.B) % four == 0 && reinterpret_cast<uintptr_t>(p.C) % four == 0;
    return dispatch(q, true, in_dtype, out_dtype, st);
}

}  // namespace kda
