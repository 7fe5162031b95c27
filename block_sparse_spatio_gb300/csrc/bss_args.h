// bss_args.h -- argument checks shared by the matrix products and the cross
// attention.  Host code only.
#pragma once
#include <cstdint>

#include "bss_block.h"
#include "bss_host.h"
#include "bss_internal.h"

namespace bss {

constexpr int64_t kMaxRowStride = int64_t(1) << 28;  // elements; a row's bytes then stay below a tensor map's limit

inline int64_t element_size(int32_t dtype) { return dtype == BSS_DTYPE_F32 ? 4 : 2; }

inline bool known_dtype(int32_t dtype) { return dtype == BSS_DTYPE_BF16 || dtype == BSS_DTYPE_F32; }

// One tensor of a call and the bytes that it touches.
struct Operand {
    const void* p = nullptr;
    const char* name = "";
    Region r;
    bool output = false;
    int over = -1;  // the input that this output may be written over, by its place in the list
};

// A [rows][width] matrix with rows `stride` elements apart (NULL: left out).
inline bss_status check_matrix(Operand* o, const void* p, const char* name, int64_t rows, int64_t stride, int64_t width,
                               int32_t dtype, bool output) {
    o->p = p;
    o->name = name;
    o->output = output;
    if (p == nullptr) return BSS_OK;
    if (!is_aligned(p, 16)) return set_error(BSS_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (rows > 1 && (stride % 8 != 0 || stride < 0 || stride > kMaxRowStride))
        return set_error(BSS_ERR_INVALID_ARG, "%s: the row stride must be a multiple of 8 elements, 0 .. 2^28", name);
    o->r = region_2d(p, rows, rows > 1 ? stride : 0, width, element_size(dtype));
    if (output && o->r.self_overlap) return set_error(BSS_ERR_INVALID_ARG, "%s: rows overlap", name);
    return BSS_OK;
}

// A run of `bytes` bytes.
inline bss_status check_run(Operand* o, const void* p, const char* name, int64_t bytes, uintptr_t alignment, bool output) {
    o->p = p;
    o->name = name;
    o->output = output;
    if (p == nullptr) return BSS_OK;
    if (!is_aligned(p, alignment)) return set_error(BSS_ERR_INVALID_ARG, "%s must be %d-byte aligned", name, (int)alignment);
    o->r = region_2d(p, 1, 0, bytes, 1);
    return BSS_OK;
}

// An output shares no byte with another tensor, but for the input that it is
// written over: the very same bytes, each read by the thread that writes it, and
// read by nothing else.
inline bss_status check_outputs(const Operand* t, int n) {
    for (int i = 0; i < n; ++i) {
        if (t[i].p == nullptr || !t[i].output) continue;
        for (int j = 0; j < n; ++j) {
            if (j == i || t[j].p == nullptr || (t[j].output && j < i)) continue;
            if (j == t[i].over && t[j].r.same_bytes(t[i].r) && !t[j].r.self_overlap) continue;
            if (!disjoint(t[i].r, t[j].r))
                return set_error(BSS_ERR_INVALID_ARG, "%s overlaps %s", t[i].name, t[j].name);
        }
    }
    return BSS_OK;
}

inline bss_status check_workspace(const void* p, int64_t bytes, int64_t need) {
    if (need > 0 && (p == nullptr || bytes < need))
        return set_error(BSS_ERR_INVALID_ARG, "workspace of %lld bytes needed (got %lld)", (long long)need,
                         (long long)(p == nullptr ? 0 : bytes));
    return BSS_OK;
}

}  // namespace bss
