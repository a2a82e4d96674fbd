// abi.h -- what the files that implement the C ABI share: the calling thread's
// error message and the carve-up of a caller's workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sk {

// The message sinkhorn_last_error() returns; fail() sets it and returns `code`.
void clear_error();
int fail(int code, const char *fmt, ...);
int hip_fail(hipError_t e, const char *where);

// Bump allocator over the caller's workspace (256-byte aligned pieces).
// Pieces of the caller's workspace, each at a 256-byte aligned address (the
// sizes add 256 bytes of slack for a workspace that starts unaligned).
struct Carve {
    char *base;
    size_t off = 0;
    template <typename T> T *take(size_t count)
    {
        const uintptr_t at = (uintptr_t)base + off;
        off += (((at + 255) & ~(uintptr_t)255) - at);
        T *p = base ? reinterpret_cast<T *>(base + off) : nullptr;
        off += count * sizeof(T);
        return p;
    }
};

}  // namespace sk
