// The compiled calls (csrc/torch_calls.cpp) without a GPU: the same source on host
// tensors, with the library's functions replaced by ones that record their arguments
// and fill their outputs.  A call that would hand the library something out of order
// shows here, where nothing follows the pointers.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <string.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ck.h"

namespace c10::cuda {
inline int host_device() { return -1; }
struct HostStream {
    void *stream() const { return nullptr; }
};
inline HostStream host_stream(int) { return {}; }
}  // namespace c10::cuda
namespace at::detail {
inline Tensor host_empty(IntArrayRef shape, ScalarType type, c10::Device, std::nullopt_t) { return at::empty(shape, type); }
}  // namespace at::detail

namespace {
int g_calls = 0;
int64_t g_ldm = 0;
constexpr int kMark = 0x5a;
ck_status called() { return ++g_calls, CK_OK; }
void fill_rows(void *p, int64_t rows, int64_t cols, int64_t ld) {
    for (int64_t i = 0; p && i < rows; ++i) memset(static_cast<uint16_t *>(p) + i * ld, kMark, cols * 2);
}
size_t tiles(ck_fp4_format f, int64_t rows, int64_t K) { return (rows + 127) / 128 * ((K + (f ? 63 : 127)) / (f ? 64 : 128)) * 512; }
}  // namespace

extern "C" {
CK_API int check_calls() { return g_calls; }
CK_API int64_t check_ldm() { return g_ldm; }

size_t ck_fp4_scale_bytes(ck_fp4_format f, int64_t rows, int64_t K) { return tiles(f, rows, K); }
size_t ck_fp4_linear_workspace_bytes(int64_t, int64_t, ck_fp4_format) { return 256; }
size_t ck_fp4_swiglu_mlp_workspace_bytes(int64_t, int64_t, int64_t, ck_fp4_format) { return 256; }
ck_status ck_fp4_quantize(const void *, ck_dtype, int64_t M, int64_t K, int64_t, ck_input_act, ck_fp4_format f, float, void *codes,
                          void *scales, ck_stream_t) {
    memset(codes, kMark, M * K / 2), memset(scales, kMark, tiles(f, M, K));
    return called();
}
ck_status ck_fp4_gemm(const void *, const void *, int64_t M, int64_t, ck_fp4_format, const void *, const void *, int64_t N, float,
                      const void *, const void *, void *y, ck_stream_t) {
    fill_rows(y, M, N, N);
    return called();
}
ck_status ck_fp4_linear(const void *, int64_t M, int64_t, int64_t, ck_input_act, ck_fp4_format, float, const void *, const void *,
                        float, int64_t N, const void *, const void *, void *y, void *, size_t, ck_stream_t) {
    fill_rows(y, M, N, N);
    return called();
}
ck_status ck_fp4_swiglu_mlp(const void *, int64_t M, int64_t H, int64_t, ck_fp4_format, float, const void *, const void *, float,
                            const void *, float, const void *, const void *, float, const void *, const void *, void *y, void *,
                            size_t, ck_stream_t) {
    fill_rows(y, M, H, H);
    return called();
}
ck_status ck_block_norm(const void *, int64_t, const void *, int64_t, int64_t T, int64_t H, const void *, const void *, const void *,
                        const void *, int64_t ldm, int64_t, float, float, ck_norm, const void *, const void *, ck_dtype, float,
                        void *h, int64_t ldh, void *n, int64_t ldn, ck_stream_t) {
    g_ldm = ldm;
    fill_rows(h, T, H, ldh), fill_rows(n, T, H, ldn);
    return called();
}
ck_status ck_block_norm_fp4(const void *, int64_t, const void *, int64_t, int64_t T, int64_t H, const void *, const void *,
                            const void *, const void *, int64_t ldm, int64_t, float, float, ck_norm, const void *, const void *,
                            ck_dtype, float, void *h, int64_t ldh, ck_fp4_format f, float, void *codes, void *scales, ck_stream_t) {
    g_ldm = ldm;
    fill_rows(h, T, H, ldh);
    memset(codes, kMark, T * H / 2), memset(scales, kMark, tiles(f, T, H));
    return called();
}
}  // extern "C"

// (the headers are in, so these words change in the source below only)
#define is_cuda is_cpu
#define current_device host_device
#define getCurrentCUDAStream host_stream
#define empty_cuda host_empty
#include "torch_calls.cpp"
