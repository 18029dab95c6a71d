// Error text of the calling thread, shared by every entry point of
// libgemm_f32.so (gemm_f32_last_error returns it).
#pragma once

namespace gemm_f32_impl {

void clear_error();

// Keeps the formatted text and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

}  // namespace gemm_f32_impl
