// kda_ssm_bwd_scan.cu -- the passes of the selective scan's gradients (kda_ssm_bwd.cu) that run along
// the sequences, as modes of the prompt's scan (kda_ssm_scan.cuh).
#include "kda_ssm_scan.cuh"

namespace kda {
namespace ssm {
namespace {

template <typename T, typename Tg>
cudaError_t run(const ScanArgs& q, cudaStream_t st) {
    const cudaError_t e = launch_scan<T, T, Scan::kKeep>(q, st);
    if (e != cudaSuccess || !q.seg_grad) return e;
    return launch_scan<T, Tg, Scan::kBack>(q, st);
}

}  // namespace

cudaError_t launch_ssm_bwd_scans(const BwdArgs& b, int in_dtype, int grad_dtype, cudaStream_t st) {
    ScanArgs q{};
    q.p = b.p;
    q.g = b.g;
    q.chunks = b.chunks;
    q.ckpt = b.ckpt;
    q.ckpt_n = 4 * lanes_for(b.p.N);
    q.vec = b.vec;
    q.vec_bc = b.vec_bc;
    q.vec_state = b.p.N % 4 == 0;  // into the workspace: 256-byte boundaries
    if (b.multi) {
        q.ckpt_dt = b.ckpt_dt;
        q.seg_state = b.seg_h;
        q.seg_dt = b.seg_dt;
        q.seg_grad = b.seg_g;
    }
    const int cw = 64 / scan_lanes(b.p.N), per_group = b.p.D / b.p.G;
    q.scan_warps = kMostScan;
    while (q.scan_warps > 1 && (q.scan_warps - 1) * cw >= per_group) --q.scan_warps;
    if (in_dtype == KDA_BF16)
        return grad_dtype == KDA_BF16 ? run<__nv_bfloat16, __nv_bfloat16>(q, st) : run<__nv_bfloat16, float>(q, st);
    return grad_dtype == KDA_BF16 ? run<float, __nv_bfloat16>(q, st) : run<float, float>(q, st);
}

}  // namespace ssm
}  // namespace kda
