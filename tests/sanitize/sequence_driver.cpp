// The sequence operators' argument checks for a build with AddressSanitizer and UndefinedBehaviorSanitizer on the host
// code: sizes at and past every limit, in every combination of extreme values, so that no check overflows on its way to
// an answer. Every call made here must be refused before any launch (or ask for a size only).
#include <climits>
#include <cstdint>
#include <cstdio>

#include "mdlstm.h"

static int g_bad = 0, g_calls = 0;
#define REFUSED(call)                                                                                  \
    do {                                                                                               \
        ++g_calls;                                                                                     \
        const int rc_ = (call);                                                                        \
        if (rc_ != MDL_EINVAL && rc_ != MDL_EOVERFLOW && rc_ != MDL_EUNSUPPORTED && rc_ != MDL_ESIZE) { \
            std::fprintf(stderr, "%s:%d: %s returned %d\n", __FILE__, __LINE__, #call, rc_);           \
            ++g_bad;                                                                                   \
        }                                                                                              \
    } while (0)

int main() {
    void* p = reinterpret_cast<void*>(uintptr_t(1) << 20);
    float* f = static_cast<float*>(p);
    const int64_t* off = static_cast<const int64_t*>(p);
    const int32_t* ids = static_cast<const int32_t*>(p);
    const int64_t big[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX / 2, int64_t(1) << 60};
    const int32_t wide[] = {INT32_MIN, -1, 0, 1, 7, INT32_MAX};
    size_t bytes = 0;
    for (int64_t T : big)
        for (int32_t D : wide) {
            REFUSED(mdl_scan_workspace_size(T, D, MDL_F32, &bytes));
            REFUSED(mdl_blocknorm_workspace_size(T, D, MDL_BF16, &bytes));
            for (int64_t ld : big) {
                REFUSED(mdl_scan_forward(off, 1, T, D, MDL_BF16, 0, p, p, p, ld, f, p, ld, f, p, SIZE_MAX, nullptr));
                REFUSED(mdl_scan_backward(off, 1, T, D, MDL_F32, 1, p, p, p, ld, f, p, ld, f, p, p, p, ld, f, p, SIZE_MAX,
                                          nullptr));
                REFUSED(mdl_blocknorm_forward(T, D, MDL_F32, p, ld, p, ld, p, ld, f, f, f, 1e-6f, p, p, ld, nullptr));
                REFUSED(mdl_blocknorm_backward(T, D, MDL_F32, p, ld, p, ld, p, ld, f, f, f, 1e-6f, p, p, ld, p, p, p, ld, f,
                                               f, f, p, SIZE_MAX, nullptr));
                REFUSED(mdl_distill(T, D, 1, MDL_F32, p, ld, ids, p, MDL_F32, f, 1.f, f, p, ld, nullptr));
            }
        }
    // strides past every limit with sizes that are fine otherwise
    for (int64_t ld : big) {
        REFUSED(mdl_scan_forward(off, 1, 10, 8, MDL_F32, 0, p, p, p, ld, f, p, 8, f, p, SIZE_MAX, nullptr));
        REFUSED(mdl_scan_forward(off, 1, 10, 8, MDL_F32, 0, p, p, p, 8, f, p, ld, f, p, SIZE_MAX, nullptr));
        REFUSED(mdl_blocknorm_forward(10, 8, MDL_F32, p, 8, p, ld, p, 8, f, f, f, 1e-6f, p, p, 8, nullptr));
        REFUSED(mdl_distill(10, 8, 2, MDL_F32, p, 8, ids, p, MDL_F32, f, 1.f, f, p, ld, nullptr));
        REFUSED(mdl_scan_step(4, 8, MDL_F32, p, p, p, ld, ids, 9, f, f, p, 8, nullptr));
    }
    for (int32_t S : wide)
        for (int32_t D : wide) {
            if (S == 1 && (D == 1 || D == 7)) continue;  // in order
            if (S == 7 && (D == 1 || D == 7)) continue;
            if ((S == 1 && D == INT32_MAX) || (S == INT32_MAX && D == 1)) continue;
            REFUSED(mdl_scan_step(S, D, MDL_F32, p, p, p, INT32_MAX, ids, S, f, f, p, INT32_MAX, nullptr));
        }
    std::printf("sequence driver: %d calls, %d failures\n", g_calls, g_bad);
    return g_bad == 0 ? 0 : 1;
}
