// Test aid: which outputs the pair kernel writes by TMA boxes, for CPU tests (the library's host source as it stands;
// the kernel launchers come from libgemm_gb300.so and are not called).
#include "../dense_gemm_epilogues_tcgen05_gb300/csrc/gemm_api.cu"

extern "C" int c_map_ok(unsigned long long base, int64_t N, int64_t ldc, int es) {
    return c_tma_ok(reinterpret_cast<const void *>(base), N, ldc, es) ? 1 : 0;
}
