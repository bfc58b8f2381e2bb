// kda_conv.cu -- the short causal convolution over each channel that stands in front of the
// recurrence, for prompts, single tokens and training.
//
//   p_t[c] = bias[c] + sum_{j<W} w[c][j] x_{t-W+1+j}[c]        y_t = p_t, or p_t sigmoid(p_t)
// with the rows before a sequence's first token taken from its state (W-1 rows, oldest first)
// or zero, and backwards, with g_t = dL/dp_t (0 past the sequence's end):
//   dx_t[c] = sum_j w[c][j] g_{t+W-1-j}[c]     dw[c][j] = sum_t g_t x_{t-W+1+j}     db[c] = sum_t g_t.
//
// Bound by HBM: every row is read once and written once, 2W + 5 operations an element.  A thread
// owns V neighbouring channels (16 bytes of bf16 or fp32; two elements or one where the sizes or
// the alignment do not allow it) and walks L tokens with the last W-1 rows in registers, so a row
// is read again only by the thread of the next L tokens (W-1 of L + W-1 rows, from L2).
//
// Measured (GB300, bf16, W = 4, SiLU): 188,232 tokens x 8192 channels 1.005 ms, 6.14 TB/s, 0.92 of the
// copy rate; gradients of 32,768 x 4096 0.193 ms, 4.2 TB/s, 0.62 of it: 20 operations an element and
// 128 registers a thread, which leave 16 warps an SM and do not hold the sums, weights and windows of 4
// channels beside a batch of rows: the variants of 4 channels spill (bytes of spill stores a thread for 4, 3
// and 2 taps: x and gradients bf16 156, 104, 48; bf16 and fp32 504, 252, 156; fp32 and bf16 396, 320, 200;
// fp32 1192, 536, 696).  That size with 4 taps: bf16 x with fp32 gradients 0.256 ms (bytes alone 0.201), fp32
// with bf16 0.238 (0.161), fp32 0.557 (0.241).  In bf16 8 channels a thread, 5 CTAs an SM and longer batches were
// slower, and 4 rows a batch too (0.208 against 0.199 then); the choice was not timed in the other types.
#include <type_traits>

#include "kda_vec.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;  // rows of a thread in flight
constexpr int kBwdBatch = 6;  // and of the gradients: a multiple of 2 and 3, so that the windows of W-1 rows turn without moves

// Row t of the sequence [a, ..) of state row base `init` as raw channels, t may lie before a.
template <typename T, int V, int W>
__device__ __forceinline__ Raw<T, V> history_row(const ConvProblem& p, const T* x, int s, int64_t a, int64_t t, int c0) {
    if (t >= a) return ld_raw<T, V>(x + t * p.x_stride + c0);
    if (p.init) {
        const int64_t j = t - a + (W - 1);
        return ld_raw<T, V>(static_cast<const T*>(p.init) + ((int64_t)s * (W - 1) + j) * p.D + c0);
    }
    Raw<T, V> z;
    memset(&z, 0, sizeof(z));
    return z;
}

// The weights of V channels, [tap][channel], and their biases, for the column blocks' threads.  Read
// straight from [D, W] a warp's load would touch 32 separate lines; so the block's weights come in
// coalesced, and each thread takes its V W + V values from shared memory, an odd number of 16-byte
// units apart, which keeps the banks apart too.  Called by every thread of the block.
template <int V, int W>
struct TapBuffer {
    static constexpr int kStride = V <= 2 ? 1 : 4 * (((V * W + V) / 4) | 1);
    float w[V <= 2 ? 1 : kThreads * kStride];
};
template <int V, int W>
__device__ __forceinline__ void load_taps(const ConvProblem& p, TapBuffer<V, W>& s, int cb, int cx, int c0,
                                          float (&w)[W][V], float (&b)[V]) {
    if constexpr (V <= 2) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = c0 + i < p.D ? __ldg(p.weight + (int64_t)(c0 + i) * W + j) : 0.f;
            b[i] = p.bias && c0 + i < p.D ? __ldg(p.bias + c0 + i) : 0.f;
        }
    } else {
        constexpr int S = TapBuffer<V, W>::kStride;
        const int first = (cb << p.log_cx) * V, n = min(V << p.log_cx, p.D - first);
        for (int i = threadIdx.x; i < n * W; i += kThreads)
            s.w[i / (V * W) * S + i % (V * W)] = __ldg(p.weight + (int64_t)first * W + i);
        for (int i = threadIdx.x; i < n; i += kThreads)
            s.w[i / V * S + V * W + i % V] = p.bias ? __ldg(p.bias + first + i) : 0.f;
        __syncthreads();
        float f[V * W + V];
#pragma unroll
        for (int i = 0; i < (V * W + V) / 4; ++i) {
            const float4 v = *reinterpret_cast<const float4*>(s.w + cx * S + 4 * i);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][i] = f[i * W + j];
            b[i] = f[V * W + i];
        }
    }
}

// The last W-1 rows of sequence s behind its initial state: its final state.
template <typename T, int V, int W>
__device__ __forceinline__ void write_final(const ConvProblem& p, int s, int c0) {
    int64_t a, e;
    seq_range(p.seqs, s, a, e);
    Raw<T, V> r[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
        r[j] = history_row<T, V, W>(p, static_cast<const T*>(p.x), s, a, e - (W - 1) + j, c0);
    T* out = static_cast<T*>(p.final_state) + (int64_t)s * (W - 1) * p.D + c0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) st_raw<T, V>(out + (int64_t)j * p.D, r[j]);
}

template <typename T, typename To, int V, int W>
__global__ void __launch_bounds__(kThreads, 4) conv_fwd_kernel(ConvProblem p) {
    if (blockIdx.x >= p.main_blocks) {  // the final states
        const int64_t i = (int64_t)(blockIdx.x - p.main_blocks) * kThreads + threadIdx.x;
        const int nv = p.D / V;
        if (i < (int64_t)p.seqs.N * nv) write_final<T, V, W>(p, (int)(i / nv), (int)(i % nv) * V);
        return;
    }
    const int cx = threadIdx.x & ((1 << p.log_cx) - 1), sub = threadIdx.x >> p.log_cx;
    const int cb = blockIdx.x % p.col_blocks;
    const int c0 = ((cb << p.log_cx) + cx) * V;
    const int64_t t0 = ((int64_t)(blockIdx.x / p.col_blocks) * (kThreads >> p.log_cx) + sub) * p.L;
    __shared__ __align__(16) TapBuffer<V, W> taps;
    float w[W][V], b[V], h[W - 1][V];
    load_taps<V, W>(p, taps, cb, cx, c0, w, b);
    if (c0 >= p.D || t0 >= p.seqs.T_total) return;
    const int64_t t1 = min(t0 + p.L, p.seqs.T_total);
    const T* x = static_cast<const T*>(p.x);
    To* y = static_cast<To*>(p.y);

    for (int64_t t = t0; t < t1;) {
        int64_t a, e;
        const int s = seq_of(p.seqs, t, a, e);
        const int64_t end = min(e, t1);
#pragma unroll
        for (int k = 0; k < W - 1; ++k) widen<T, V>(history_row<T, V, W>(p, x, s, a, t - (W - 1) + k, c0), h[k]);
        auto load = [&](int64_t from, Raw<T, V>(&r)[kBatch], int n) {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (i < n) r[i] = ld_raw<T, V>(x + (from + i) * p.x_stride + c0);
        };
        auto rows = [&](const Raw<T, V>(&r)[kBatch], auto count) {
            constexpr int n = decltype(count)::value;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                float f[V], o[V];
                widen<T, V>(r[i], f);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float acc = b[v];
#pragma unroll
                    for (int k = 0; k < W - 1; ++k) acc = fmaf(w[k][v], h[k][v], acc);
                    o[v] = fmaf(w[W - 1][v], f[v], acc);
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; ++k) h[k][v] = h[k + 1][v];
                    h[W - 2][v] = f[v];
                }
                if (p.act == KDA_ACT_SILU)  // one branch a row: the channels' chains overlap
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] *= sigmoid(o[v]);
                st_vec<V>(y + (t + i) * p.D + c0, o);
            }
            t += n;
        };
        // kBatch rows at a time, the next ones on the way while these are worked on
        Raw<T, V> cur[kBatch], next[kBatch];
        if (t + kBatch <= end) load(t, cur, kBatch);
        while (t + kBatch <= end) {
            if (t + 2 * kBatch <= end) load(t + kBatch, next, kBatch);
            rows(cur, std::integral_constant<int, kBatch>{});
#pragma unroll
            for (int i = 0; i < kBatch; ++i) cur[i] = next[i];
        }
        while (t < end) {
            load(t, cur, 1);
            rows(cur, std::integral_constant<int, 1>{});
        }
    }
}

// One token per session, the state moved on in place.  A thread takes L sessions of its channels, two at a
// time: the next two are loaded into the registers of the last ones, so their latency is waited for.  256 sessions
// of 12,288 channels: four such rounds at 10 warps an SM, 13 us with cold inputs against 7.6 for the bytes.
template <typename T, typename To, int V, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvProblem p) {
    constexpr int kSess = 2;  // in flight
    const int cx = threadIdx.x & ((1 << p.log_cx) - 1), sub = threadIdx.x >> p.log_cx;
    const int cb = blockIdx.x % p.col_blocks;
    const int c0 = ((cb << p.log_cx) + cx) * V;
    const int64_t s0 = ((int64_t)(blockIdx.x / p.col_blocks) * (kThreads >> p.log_cx) + sub) * p.L;
    const int64_t s1 = min(s0 + p.L, (int64_t)p.seqs.N);
    __shared__ __align__(16) TapBuffer<V, W> taps;
    Raw<T, V> r[kSess][W];
    auto rows = [&](int64_t s) { return static_cast<T*>(p.final_state) + s * (W - 1) * p.D + c0; };
    auto load = [&](int64_t s) {
#pragma unroll
        for (int i = 0; i < kSess; ++i)
            if (c0 < p.D && s + i < s1) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) r[i][j] = ld_raw<T, V>(rows(s + i) + (int64_t)j * p.D);
                r[i][W - 1] = ld_raw<T, V>(static_cast<const T*>(p.x) + (s + i) * p.x_stride + c0);
            }
    };
    load(s0);  // on the way while the weights come
    float w[W][V], b[V];
    load_taps<V, W>(p, taps, cb, cx, c0, w, b);
    if (c0 >= p.D) return;
    for (int64_t s = s0; s < s1; s += kSess) {
#pragma unroll
        for (int i = 0; i < kSess; ++i)
            if (s + i < s1) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = b[v];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    float f[V];
                    widen<T, V>(r[i][j], f);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] = fmaf(w[j][v], f[v], o[v]);
                }
                if (p.act == KDA_ACT_SILU)
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] *= sigmoid(o[v]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) st_raw<T, V>(rows(s + i) + (int64_t)j * p.D, r[i][j + 1]);
                st_vec<V>(static_cast<To*>(p.y) + (s + i) * p.D + c0, o);
            }
        load(s + kSess);
    }
}

// Gradients.  A thread walks its L tokens and W-1 more (whose g reaches back into them), with the
// sums of the last W rows of dx in registers; row t leaves when g_{t+W-1} has been added.  The
// rows of d_init belong to the thread that holds the sequence's first token.  Its sums for dw and
// db go to partial[token piece][tap or bias][channel] and are added in order by a second kernel.
template <typename T, typename Tg, int V, int W>
__global__ void __launch_bounds__(kThreads, 4) conv_bwd_kernel(ConvProblem p) {
    const T* x = static_cast<const T*>(p.x);
    if (blockIdx.x >= p.main_blocks) {  // d_init of the sequences without a token
        const int nv = p.D / V;
        const int64_t i = (int64_t)(blockIdx.x - p.main_blocks) * kThreads + threadIdx.x;
        if (i >= (int64_t)p.seqs.N * nv) return;
        const int s = (int)(i / nv), c0 = (int)(i % nv) * V;
        int64_t a, e;
        seq_range(p.seqs, s, a, e);
        if (e > a) return;
        for (int j = 0; j < W - 1; ++j)
            for (int v = 0; v < V; ++v) {
                const int64_t o = ((int64_t)s * (W - 1) + j) * p.D + c0 + v;
                p.d_init[o] = p.d_final ? p.d_final[o] : 0.f;
            }
        return;
    }
    const int cx = threadIdx.x & ((1 << p.log_cx) - 1), sub = threadIdx.x >> p.log_cx;
    const int cb = blockIdx.x % p.col_blocks;
    const int c0 = ((cb << p.log_cx) + cx) * V;
    const int64_t piece = (int64_t)(blockIdx.x / p.col_blocks) * (kThreads >> p.log_cx) + sub;
    const int64_t t0 = piece * p.L;
    __shared__ __align__(16) TapBuffer<V, W> taps;
    float w[W][V], b[V], h[W - 1][V], dw[W][V], db[V];
    load_taps<V, W>(p, taps, cb, cx, c0, w, b);
    if (c0 >= p.D || t0 >= p.seqs.T_total) return;
    const int64_t t1 = min(t0 + p.L, p.seqs.T_total);
    const Tg* dy = static_cast<const Tg*>(p.d_out);
    Tg* dx = static_cast<Tg*>(p.dx);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }

    for (int64_t first = t0; first < t1;) {
        int64_t a, e;
        const int s = seq_of(p.seqs, first, a, e);
        const int64_t end = min(e, t1);       // own tokens: [first, end)
        const int64_t live = min(e, end + W - 1);  // tokens whose g is wanted
        float acc[W][V];                      // acc[k]: dx of row t - (W-1) + k
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k][v] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) widen<T, V>(history_row<T, V, W>(p, x, s, a, first - (W - 1) + k, c0), h[k]);

        // kBwdBatch tokens from t.  kInside: all of them own, and the rows that they complete too (the
        // common case, without a test in it).
        auto batch = [&](int64_t t, auto inside) {
            constexpr bool kInside = decltype(inside)::value;
            Raw<T, V> rx[kBwdBatch];
            Raw<Tg, V> rg[kBwdBatch];
#pragma unroll
            for (int i = 0; i < kBwdBatch; ++i)
                if (kInside || t + i < live) {
                    rx[i] = ld_raw<T, V>(x + (t + i) * p.x_stride + c0);
                    rg[i] = ld_raw<Tg, V>(dy + (t + i) * p.D + c0);
                }
#pragma unroll
            for (int i = 0; i < kBwdBatch; ++i) {
                const int64_t tt = t + i;
                if (kInside || tt < live) {
                    float f[V], g[V];
                    widen<T, V>(rx[i], f);
                    widen<Tg, V>(rg[i], g);
                    if (p.act == KDA_ACT_SILU)  // one branch a row: the channels' chains overlap
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            float z = b[v];
#pragma unroll
                            for (int k = 0; k < W - 1; ++k) z = fmaf(w[k][v], h[k][v], z);
                            z = fmaf(w[W - 1][v], f[v], z);
                            const float sg = sigmoid(z);
                            g[v] *= sg * fmaf(z, 1.f - sg, 1.f);
                        }
                    if (kInside || tt < end)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            db[v] += g[v];
                            dw[W - 1][v] = fmaf(g[v], f[v], dw[W - 1][v]);
#pragma unroll
                            for (int k = 0; k < W - 1; ++k) dw[k][v] = fmaf(g[v], h[k][v], dw[k][v]);
                        }
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int k = 0; k < W; ++k) acc[k][v] = fmaf(w[k][v], g[v], acc[k][v]);
#pragma unroll
                        for (int k = 0; k + 1 < W - 1; ++k) h[k][v] = h[k + 1][v];
                        h[W - 2][v] = f[v];
                    }
                }
                // row r has all its terms now (or, past `live`, will get no more)
                const int64_t r = tt - (W - 1);
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = acc[0][v];
                if constexpr (kInside) {
                    st_vec<V>(dx + r * p.D + c0, o);
                } else {
                    const bool mine = r >= first ? r < end : (first == a && p.d_init != nullptr && r >= a - (W - 1));
                    if (mine && tt < end + W - 1) {
                        const int64_t j = r - (e - (W - 1));  // its row of the final state
                        if (p.d_final && j >= 0)
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                o[v] += p.d_final[((int64_t)s * (W - 1) + j) * p.D + c0 + v];
                        if (r >= a) {
                            st_vec<V>(dx + r * p.D + c0, o);
                        } else {
                            float* di = p.d_init + ((int64_t)s * (W - 1) + (r - a + W - 1)) * p.D + c0;
#pragma unroll
                            for (int v = 0; v < V; ++v) di[v] = o[v];
                        }
                    }
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
#pragma unroll
                    for (int k = 0; k + 1 < W; ++k) acc[k][v] = acc[k + 1][v];
                    acc[W - 1][v] = 0.f;
                }
            }
        };
        int64_t t = first;
        batch(t, std::false_type{});  // kBwdBatch >= W - 1: the rows before `first` end here
        for (t += kBwdBatch; t + kBwdBatch <= end; t += kBwdBatch) batch(t, std::true_type{});
        for (; t < end + W - 1; t += kBwdBatch) batch(t, std::false_type{});
        first = end;
    }
    float* part = p.partial + piece * (W + 1) * p.D + c0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[(int64_t)j * p.D + v] = dw[j][v];
        part[(int64_t)W * p.D + v] = db[v];
    }
}

// dw[c][j] and db[c]: the pieces' sums, added in a fixed order.  Block (32, n): 32 channels of one
// tap; n runs of pieces side by side, 8, or 32 where the pieces are many (32 cost 6 us more at 76
// pieces, and 16 us less at 2210).
__global__ void __launch_bounds__(1024) conv_bwd_sum_kernel(const float* partial, int64_t pieces, int D, int W,
                                                           float* dweight, float* dbias) {
    __shared__ float s[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x, j = blockIdx.y;
    const int64_t per = (pieces + blockDim.y - 1) / blockDim.y;
    const int64_t lo = per * threadIdx.y, hi = min(lo + per, pieces);
    float sum = 0.f;
    if (c < D)
#pragma unroll 8
        for (int64_t i = lo; i < hi; ++i) sum += partial[(i * (W + 1) + j) * D + c];
    s[threadIdx.y][threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
        for (int k = 1; k < blockDim.y; ++k) sum += s[k][threadIdx.x];
        if (j < W) dweight[(int64_t)c * W + j] = sum;
        else if (dbias) dbias[c] = sum;
    }
}

// Rows per thread: at most `longest` (the W-1 rows read twice, the weights and the partial sums weigh
// little then), and so many pieces that `ctas` CTAs an SM are filled a whole number of times; at least 4.
int rows_per_thread(int64_t rows, int64_t row_threads, int longest, int ctas = 4) {
    const int64_t wave = 152ll * ctas * kThreads / row_threads;  // pieces that the chip holds at once
    const int64_t pieces = wave > 1 ? wave : 1;
    int64_t L = (rows + pieces - 1) / pieces;
    if (L > longest) {
        const int64_t waves = (L + longest - 1) / longest;
        L = (rows + pieces * waves - 1) / (pieces * waves);
    }
    return L < 4 ? 4 : (int)L;
}

// The gradients', the same for whatever vector width: the workspace is sized by it.
int bwd_rows(int64_t T_total, int D) { return rows_per_thread(T_total, (D + 3) / 4, 512); }

// Columns of threads: a row's vectors are spread over up to 128.
void plan(ConvProblem& p, int V, int L) {
    const int nv = (p.D + V - 1) / V;
    p.log_cx = 0;
    while (p.log_cx < 7 && (1 << p.log_cx) < nv) ++p.log_cx;
    p.col_blocks = (nv + (1 << p.log_cx) - 1) >> p.log_cx;
    p.L = L;
}

int64_t pieces_of(int64_t T_total, int L) { return (T_total + L - 1) / L; }

template <typename T>
bool vector_ok(const ConvProblem& p, int V) {
    const uintptr_t bytes = V * sizeof(T);
    auto ok = [&](const void* q) { return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0; };
    return p.D % V == 0 && p.x_stride % V == 0 && ok(p.x) && ok(p.init) && ok(p.final_state);
}
bool out_ok(const void* q, int bytes) { return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0; }

template <typename T, typename To, int V, int W>
cudaError_t fwd_vw(ConvProblem p, bool step, cudaStream_t st) {
    const int64_t state_items = (int64_t)p.seqs.N * (p.D / V);
    const int64_t state_blocks = (state_items + kThreads - 1) / kThreads;
    if (step) {  // here the tokens are the sessions
        // 8 sessions a thread, fewer while that leaves SMs with less than 256 threads
        int L = 8;
        while (L > 1 && pieces_of(p.seqs.N, L) * (p.D / V) < 152 * 256) L >>= 1;
        plan(p, V, L);
        const int subs = kThreads >> p.log_cx;
        const int64_t blocks = (pieces_of(p.seqs.N, p.L) + subs - 1) / subs * p.col_blocks;
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        conv_step_kernel<T, To, V, W><<<(unsigned)blocks, kThreads, 0, st>>>(p);
        return cudaGetLastError();
    }
    // 4 CTAs an SM fit the registers of 16-byte vectors; narrow ones take fewer and want more threads
    plan(p, V, rows_per_thread(p.seqs.T_total, p.D / V, 128, V <= 2 ? 8 : 4));
    const int subs = kThreads >> p.log_cx;
    const int64_t main_blocks = (pieces_of(p.seqs.T_total, p.L) + subs - 1) / subs * p.col_blocks;
    const int64_t tail = p.final_state ? state_blocks : 0;
    if (main_blocks + tail > INT32_MAX) return cudaErrorInvalidValue;
    p.main_blocks = (unsigned)main_blocks;
    // A final state written over the initial one: only after every row has read it.
    const bool apart = p.final_state && p.final_state == p.init && main_blocks > 0;
    const unsigned grid = (unsigned)(main_blocks + (apart ? 0 : tail));
    if (grid) conv_fwd_kernel<T, To, V, W><<<grid, kThreads, 0, st>>>(p);
    if (apart) {
        p.main_blocks = 0;
        conv_fwd_kernel<T, To, V, W><<<(unsigned)tail, kThreads, 0, st>>>(p);
    }
    return cudaGetLastError();
}

template <typename T, typename To, int V>
cudaError_t fwd_v(const ConvProblem& p, bool step, cudaStream_t st) {
    switch (p.W) {
        case 2: return fwd_vw<T, To, V, 2>(p, step, st);
        case 3: return fwd_vw<T, To, V, 3>(p, step, st);
        default: return fwd_vw<T, To, V, 4>(p, step, st);
    }
}

template <typename T, typename To>
cudaError_t fwd_t(const ConvProblem& p, bool step, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    if (vector_ok<T>(p, V) && out_ok(p.y, 16)) return fwd_v<T, To, V>(p, step, st);
    if (vector_ok<T>(p, 2) && out_ok(p.y, 2 * sizeof(To))) return fwd_v<T, To, 2>(p, step, st);
    return fwd_v<T, To, 1>(p, step, st);
}

template <typename T, typename Tg, int V, int W>
cudaError_t bwd_vw(ConvProblem p, cudaStream_t st) {
    plan(p, V, bwd_rows(p.seqs.T_total, p.D));
    const int subs = kThreads >> p.log_cx;
    const int64_t pieces = pieces_of(p.seqs.T_total, p.L);
    const int64_t main_blocks = (pieces + subs - 1) / subs * p.col_blocks;
    const int64_t tail = p.d_init ? ((int64_t)p.seqs.N * (p.D / V) + kThreads - 1) / kThreads : 0;
    if (main_blocks + tail > INT32_MAX) return cudaErrorInvalidValue;
    p.main_blocks = (unsigned)main_blocks;
    if (main_blocks + tail) conv_bwd_kernel<T, Tg, V, W><<<(unsigned)(main_blocks + tail), kThreads, 0, st>>>(p);
    conv_bwd_sum_kernel<<<dim3((p.D + 31) / 32, W + 1), dim3(32, pieces < 512 ? 8 : 32), 0, st>>>(p.partial, pieces, p.D, W, p.dweight,
                                                                           p.dbias);
    return cudaGetLastError();
}

template <typename T, typename Tg, int V>
cudaError_t bwd_v(const ConvProblem& p, cudaStream_t st) {
    switch (p.W) {
        case 2: return bwd_vw<T, Tg, V, 2>(p, st);
        case 3: return bwd_vw<T, Tg, V, 3>(p, st);
        default: return bwd_vw<T, Tg, V, 4>(p, st);
    }
}

template <typename T, typename Tg>
cudaError_t bwd_t(const ConvProblem& p, cudaStream_t st) {
    // 4 channels: the sums and windows of 8 would take more registers than they save loads
    constexpr int V = 4;
    if (vector_ok<T>(p, V) && out_ok(p.d_out, V * sizeof(Tg)) && out_ok(p.dx, V * sizeof(Tg)))
        return bwd_v<T, Tg, V>(p, st);
    if (vector_ok<T>(p, 2) && out_ok(p.d_out, 2 * sizeof(Tg)) && out_ok(p.dx, 2 * sizeof(Tg)))
        return bwd_v<T, Tg, 2>(p, st);
    return bwd_v<T, Tg, 1>(p, st);
}

}  // namespace

cudaError_t launch_conv(const ConvProblem& p, bool step, int in_dtype, int out_dtype, cudaStream_t st) {
    if (in_dtype == KDA_BF16)
        return out_dtype == KDA_BF16 ? fwd_t<__nv_bfloat16, __nv_bfloat16>(p, step, st)
                                     : fwd_t<__nv_bfloat16, float>(p, step, st);
    return out_dtype == KDA_BF16 ? fwd_t<float, __nv_bfloat16>(p, step, st) : fwd_t<float, float>(p, step, st);
}

cudaError_t launch_conv_bwd(const ConvProblem& p, int in_dtype, int grad_dtype, cudaStream_t st) {
    if (in_dtype == KDA_BF16)
        return grad_dtype == KDA_BF16 ? bwd_t<__nv_bfloat16, __nv_bfloat16>(p, st) : bwd_t<__nv_bfloat16, float>(p, st);
    return grad_dtype == KDA_BF16 ? bwd_t<float, __nv_bfloat16>(p, st) : bwd_t<float, float>(p, st);
}

size_t conv_bwd_workspace(int64_t T_total, int D, int W) {
    return (size_t)pieces_of(T_total, bwd_rows(T_total, D)) * (W + 1) * D * sizeof(float);
}

}  // namespace kda
