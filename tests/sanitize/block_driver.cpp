// The argument checks of linear attention, dropout and the vocabulary's cross entropy for a build with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code: sizes at and past every limit, in every combination of extreme values, so
// that no check overflows on its way to an answer. Every call made here must be refused before any launch (or ask for a
// size only).
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
// answered or refused, with no overflow on the way
#define ANSWERED(call)     \
    do {                   \
        ++g_calls;         \
        (void)(call);      \
    } while (0)

static void* at(int n) { return reinterpret_cast<void*>((uintptr_t(1) << 40) * (n + 1)); }
static float* fl(int n) { return static_cast<float*>(at(n)); }

int main() {
    const int64_t* off = static_cast<const int64_t*>(at(0));
    const int32_t* ids = static_cast<const int32_t*>(at(1));
    const uint64_t* rng = static_cast<const uint64_t*>(at(2));
    const int64_t big[] = {INT64_MIN, -1, INT64_MAX, INT64_MAX / 2, int64_t(1) << 60};
    const int64_t some[] = {0, 1, 255, 1 << 20, (int64_t(1) << 33) + 1, (int64_t(1) << 36) - 1};
    const int32_t wide[] = {INT32_MIN, -1, 0, 1, 7, 128, 129, 65536, INT32_MAX};
    size_t bytes = 0;
    for (int64_t T : big)
        for (int32_t H : wide)
            for (int32_t D : wide) {
                REFUSED(mdl_linattn_workspace_size(H, T, 2, D, D, MDL_F32, &bytes));
                REFUSED(mdl_linattn_forward(off, H, T, H, D, 7, MDL_BF16, 0, fl(1), 1.f, at(2), T, at(3), T, at(4), T, fl(5),
                                            at(6), T, fl(7), at(8), SIZE_MAX, nullptr));
                REFUSED(mdl_linattn_backward(off, H, T, H, 7, D, MDL_F32, 1, fl(1), 1.f, at(2), T, at(3), T, at(4), T, fl(5),
                                             at(6), T, fl(7), at(8), T, at(9), T, at(10), T, fl(11), at(12), SIZE_MAX,
                                             nullptr));
                REFUSED(mdl_linattn_step(H, 2, D, D, MDL_F32, fl(1), 1.f, at(2), T, at(3), T, at(4), T, ids, H, fl(6), fl(6),
                                         at(7), T == INT64_MAX ? -1 : T, nullptr));
                REFUSED(mdl_dropout(T, D, MDL_F32, at(3), T, at(4), T, 0.5f, rng, at(5), T, nullptr));
                REFUSED(mdl_vocab_loss_workspace_size(T, H, D, MDL_BF16, 1, &bytes));
                REFUSED(mdl_vocab_loss(T, H, D, MDL_F32, at(3), T, at(4), ids, fl(5), fl(6), at(7), T, at(8), at(9), SIZE_MAX,
                                       nullptr));
            }
    for (int64_t T : some)
        for (int32_t H : wide)
            for (int32_t D : wide) {
                ANSWERED(mdl_linattn_workspace_size(D, T, H, 128, 7, MDL_F32, &bytes));
                ANSWERED(mdl_vocab_loss_workspace_size(T, H, D, MDL_BF16, 1, &bytes));
                ANSWERED(mdl_vocab_loss_workspace_size(T, D, H, MDL_F32, 0, &bytes));
                // no workspace where one is needed, or a stride below its row: refused whatever the sizes
                REFUSED(mdl_linattn_forward(off, H, T, H, D, 128, MDL_BF16, 0, fl(1), 1.f, at(2), -1, at(3), -1, at(4), -1,
                                            fl(5), at(6), -1, fl(7), at(8), SIZE_MAX, nullptr));
                REFUSED(mdl_linattn_backward(off, H, T, H, 128, D, MDL_F32, 1, fl(1), 1.f, at(2), -1, at(3), -1, at(4), -1,
                                             fl(5), at(6), -1, fl(7), at(8), -1, at(9), -1, at(10), -1, fl(11), at(12),
                                             SIZE_MAX, nullptr));
                REFUSED(mdl_vocab_loss(T, H, D, MDL_F32, at(3), -1, at(4), ids, fl(5), fl(6), at(7), 1, at(8), at(9), 0,
                                       nullptr));
                REFUSED(mdl_dropout(T, D, MDL_F32, at(3), -1, at(4), 1, 0.5f, rng, at(5), 1, nullptr));
            }
    std::printf("block driver: %d calls, %d failures\n", g_calls, g_bad);
    return g_bad == 0 ? 0 : 1;
}
