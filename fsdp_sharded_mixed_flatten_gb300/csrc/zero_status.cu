// The calling thread's status of the C ABI (zero_last_error) and the checked
// CUDA call.
#include "zero_status.cuh"

#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "zero_flat.h"

namespace zf {

namespace {
thread_local char g_err[512] = "";
}

int fail(int code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

int ok() {
    g_err[0] = '\0';
    return ZERO_OK;
}

int cuda_status(cudaError_t e, const char* what) {
    if (e != cudaSuccess)
        return fail(ZERO_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
    return ok();
}

bool injected(const char* what) {
    const char* v = std::getenv("ZERO_INJECT_FAILURE");
    return v != nullptr && v[0] != '\0' && std::strstr(what, v) != nullptr;
}

int injected_failure(const char* what) {
    return fail(ZERO_ERR_CUDA, "%s: injected failure", what);
}

}  // namespace zf

ZERO_API const char* zero_last_error(void) { return zf::g_err; }
