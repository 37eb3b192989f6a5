// Host-only stand-ins for the launchers of the expert feed-forward kernels:
// each checks that the arguments the host code computed are consistent and
// counts the call; nothing touches the pointers.
#include <cstdio>
#include <cstdlib>

#include "expert_kernels.h"

namespace moe {

int g_gemm = 0, g_wgrad = 0, g_stream = 0, g_mxfp4 = 0, g_pack = 0;

static void require(bool ok, const char* what) {
    if (!ok) {
        std::fprintf(stderr, "stub: inconsistent launch arguments: %s\n", what);
        std::abort();
    }
}

int64_t expert_gemm_grid(const ExpertGemmArgs& a) { return a.max_rows + a.feats; }
hipError_t launch_expert_gemm(const ExpertGemmArgs& a, hipStream_t) {
    require(a.E >= 1 && a.max_rows >= 1 && a.red % 8 == 0 && a.feats % 8 == 0 && a.out, "gemm");
    require(a.op != ExpertOp::kGatedGrad || a.pre, "gate gradient without its input");
    ++g_gemm;
    return hipSuccess;
}
int64_t expert_wgrad_grid(const ExpertWgradArgs& a) { return a.E; }
hipError_t launch_expert_wgrad(const ExpertWgradArgs& a, hipStream_t) {
    require(a.E >= 1 && a.max_rows >= 0 && a.N % 8 == 0 && a.K % 8 == 0 && a.dw, "wgrad");
    ++g_wgrad;
    return hipSuccess;
}
static void check_stream(const ExpertStreamArgs& a) {
    require(a.E >= 1 && a.max_rows >= 1 && a.red % (a.mxfp4 ? 32 : 8) == 0 &&
                a.feats % (a.mxfp4 && a.gated ? 16 : 8) == 0 && a.out && (!a.mxfp4 || !a.pre),
            "stream");
}
int64_t expert_stream_grid(const ExpertStreamArgs& a) { return a.max_rows + a.feats; }
hipError_t launch_expert_stream(const ExpertStreamArgs& a, hipStream_t) {
    check_stream(a);
    ++g_stream;
    return hipSuccess;
}
int64_t expert_mxfp4_grid(const ExpertStreamArgs& a) { return a.max_rows + a.feats; }
hipError_t launch_expert_mxfp4(const ExpertStreamArgs& a, hipStream_t) {
    check_stream(a);
    ++g_mxfp4;
    return hipSuccess;
}
hipError_t launch_pack_mxfp4(const PackMxfp4Args& a, hipStream_t) {
    require(a.K % 32 == 0 && a.N % 8 == 0, "pack");
    ++g_pack;
    return hipSuccess;
}

}  // namespace moe
