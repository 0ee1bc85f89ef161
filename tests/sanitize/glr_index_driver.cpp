// Host-only sanitizer driver (AddressSanitizer + UndefinedBehaviorSanitizer) of
// the index arithmetic that the gated linear recurrence's kernels run
// (glr_index.h), at every edge of the sizes the header allows.
#include <cstdint>
#include <cstdio>

#include "glr_index.h"
#include "glr_plan.h"

static int failures = 0;
#define EXPECT(cond)                                                              \
    do {                                                                          \
        if (!(cond)) {                                                            \
            if (++failures < 20) std::fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
        }                                                                         \
    } while (0)

// Every address of a wave's loads lies in its rows, whether or not the scalar
// offset counts for a resource's bounds check; what the check drops, it drops
// either way.
static void rows()
{
    for (int64_t D : {1, 2, 63, 64, 77, 1001, 4096, 8191, (1 << 24) - 2, (1 << 24) - 1})
        for (int size : {2, 4})
            for (int n = 0; n <= glr::kScanTokens; ++n) {
                const uint64_t row = D * size, bytes = n * row;
                const glr::RowSpan s(n, (unsigned)row);
                EXPECT(bytes < glr::kNowhere);
                for (int k = 0; k < glr::kScanTokens; ++k) {
                    const uint64_t at = s.at(k);
                    EXPECT(k >= n || at == k * row);
                    // a row's last channel
                    EXPECT(n ? at + row <= bytes : at == 0);
                    // a lane without a channel: past the resource with and without `at`, and no wrap
                    EXPECT(glr::kNowhere >= bytes && glr::kNowhere + at <= UINT32_MAX && glr::kNowhere >= bytes - at);
                }
            }
}

int main()
{
    rows();
    if (failures) return 1;
    std::printf("sanitized index checks of the linear recurrence passed\n");
    return 0;
}
