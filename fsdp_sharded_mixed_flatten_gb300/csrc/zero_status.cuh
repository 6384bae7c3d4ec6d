// Status reporting shared by the translation units of the C ABI: the calling
// thread's error message and the one way CUDA calls are made, so that every
// entry point reports and injects failures alike.
#pragma once

#include <cstdarg>

#include <cuda_runtime.h>

#define ZERO_API extern "C" __attribute__((visibility("default")))

namespace zf {

// Set the calling thread's message and return `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear it and return ZERO_OK.
int ok();

// The status of a CUDA call, with its label as the message on failure.
int cuda_status(cudaError_t e, const char* what);

// Host-side failure injection for tests of the error paths: while the
// environment variable ZERO_INJECT_FAILURE is set, a CUDA call (a launch, a
// copy, a stream ordering) whose label contains its value is not made, and
// the entry point returns ZERO_ERR_CUDA as it would for a failed call.  Read
// at every call.
bool injected(const char* what);

// One CUDA call with its status converted, unless a test injects its failure.
int injected_failure(const char* what);
template <class F>
int cuda_call(const char* what, F&& call) {
    if (injected(what)) return injected_failure(what);
    return cuda_status(call(), what);
}

}  // namespace zf
