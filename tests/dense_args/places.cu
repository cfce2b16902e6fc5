// The dense calls of the C ABI with their launches replaced (the linker's --wrap): prints where in the buffers of a
// call the kernels would be sent. Host only: the addresses are made up, nothing is launched or dereferenced.
//   places M F   ->  gated block: bytes from `saved` to the lower plane that the forward call would write, and to the
//                    one that the backward call would read
#include <cstdio>
#include <cstdlib>

#include "launch.h"
#include "linattn.h"

static int g_word;
static la::DenseArgs g_forward;
static la::GatedGradArgs g_backward;

extern "C" {
cudaError_t __wrap_cudaGetDevice(int *dev) {
    *dev = 0;
    return cudaSuccess;
}
cudaError_t __wrap_cudaGetSymbolAddress(void **p, const void *) {
    *p = &g_word;
    return cudaSuccess;
}
// la::launch_dense, la::launch_gated_grad, la::launch_dense_pair
cudaError_t __wrap__ZN2la12launch_denseERKNS_9DenseArgsEP11CUstream_st(const la::DenseArgs &a, cudaStream_t) {
    g_forward = a;
    return cudaSuccess;
}
cudaError_t __wrap__ZN2la17launch_gated_gradERKNS_13GatedGradArgsEP11CUstream_st(const la::GatedGradArgs &a, cudaStream_t) {
    g_backward = a;
    return cudaSuccess;
}
cudaError_t __wrap__ZN2la17launch_dense_pairERKNS_9DenseArgsES2_P11CUstream_st(const la::DenseArgs &, const la::DenseArgs &, cudaStream_t) {
    return cudaSuccess;
}
}

int main(int, char **argv) {
    const int M = atoi(argv[1]), F = atoi(argv[2]), K = 8;
    const int64_t ldf = ((int64_t)F + 7) / 8 * 8;
    auto at = [](int n) { return reinterpret_cast<char *>((uintptr_t)n << 53); };
    const size_t kept = la_gated_ffn_saved_bytes(M, F), room = la_gated_ffn_backward_workspace_bytes(M, F, K);
    int rc = la_gated_ffn(at(1), at(2), at(3), at(4), at(5), kept, M, F, K, K, K, K, ldf, LA_ACT_SILU, 0);
    if (!rc)
        rc = la_gated_ffn_backward(at(1), at(2), at(3), at(5), kept, at(4), at(6), at(7), at(8), M, F, K, K, K, K, ldf, K, K, K,
                                   LA_ACT_SILU, at(9), room, 0);
    if (rc) {
        printf("refused: %s\n", la_last_error());
        return 1;
    }
    printf("%zu %lld %lld\n", kept, (long long)(static_cast<char *>(g_forward.lower) - at(5)),
           (long long)(static_cast<const char *>(g_backward.lower) - at(5)));
    return 0;
}
