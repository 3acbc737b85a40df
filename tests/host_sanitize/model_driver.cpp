// Host driver for the sanitizer build of the entry points around the verification: workspace sizes
// over their whole argument ranges, the frequencies (output at its exact length), and argument checks,
// which return before any launch.  Any sanitizer report or unexpected return code is a failure.
#include <cmath>
#include <cstdio>
#include <vector>

#include "specverify.h"

static int fails = 0, checks = 0;
#define EXPECT(what, want)                                                                        \
    do {                                                                                          \
        const long long got_ = (long long)(what), want_ = (long long)(want);                      \
        ++checks;                                                                                 \
        if (got_ != want_) {                                                                      \
            std::printf("line %d: %s gave %lld, expected %lld\n", __LINE__, #what, got_, want_);  \
            ++fails;                                                                              \
        }                                                                                         \
    } while (0)

int main() {
    const int most = 0x7fffffff;
    void* fake = reinterpret_cast<void*>(0x1000);
    int32_t* fi = static_cast<int32_t*>(fake);
    float* ff = static_cast<float*>(fake);
    // workspace sizes: no overflow anywhere, zero exactly where the sizes are refused
    for (int B : {-most, -1, 0, 1, 16, 70000, 1 << 24, most})
        for (int V : {-1, 0, 1, 2048, 8192, 8193, 151936, 1 << 30, 0x7fff0000, most}) {
            const size_t n = spec_verify_probs_workspace_bytes(B, V);
            if (B < 1 || V < 1 || V == most) EXPECT(n, 0);
            ++checks;
        }
    for (int R : {-1, 0, 1, 592, 1 << 20, most})
        for (int G : {-1, 0, 1, 64, 1 << 23, most})
            for (int Hq : {0, 1, 32, 65536, most})
                for (int H : {0, 1, 8, most})
                    for (int D : {0, 8, 12, 64, 128, 256, 264, most})
                        for (long long P : {-1ll, 0ll, 1ll, 131072ll, 0x7fff0000ll, 0x7fffffffll, 1ll << 40})
                            for (int S : {-1, 0, 1, most}) {
                                const size_t n = spec_prefix_attention_workspace_bytes(R, G, Hq, H, D, P, S);
                                if (R < 0 || G < 1 || H < 1 || Hq < H || D < 8 || D > 256 || D % 8 || P < 0 || P > 0x7fff0000ll || S < 0)
                                    EXPECT(n, 0);
                                ++checks;
                            }
    // frequencies
    for (int rot = -2; rot <= 1030; ++rot)
        for (double high : {0.5, 1.0, 4.0, (double)INFINITY}) {
            std::vector<double> out(rot > 0 ? rot / 2 : 0);
            const int rc = spec_rope_frequencies(rot, 1e4, 8.0, 1.0, high, 4096, rot > 1 ? out.data() : nullptr);
            EXPECT(rc, rot >= 2 && rot % 2 == 0 && rot <= 1024 && high >= 1.0 ? SPEC_OK : SPEC_EINVAL);
            if (rc == SPEC_OK)
                for (double f : out) EXPECT(f > 0.0 && f <= 1.0, 1);
        }
    for (double bad : {0.0, -1.0, (double)NAN, (double)INFINITY}) {
        double f[4];
        EXPECT(spec_rope_frequencies(8, bad, 1.0, 1.0, 4.0, 10, f), SPEC_EINVAL);
        if (bad != 1.0) EXPECT(spec_rope_frequencies(8, 1e4, bad == -1.0 ? 0.99 : bad, 1.0, 4.0, 10, f), SPEC_EINVAL);
    }
    // argument checks
    spec_kv_cache c{fake, fake, SPEC_BF16, 4, 16, 2, 64, 2048, 128, 64, nullptr, nullptr};
    for (int T : {-1, 1 << 24, most})
        EXPECT(spec_kv_append(fake, 256, 64, fake, 256, 64, fake, 128, 64, fake, 128, 64, SPEC_BF16, T, 4, 2, 64, fi, fi,
                              static_cast<double*>(fake), 64, 1.0f, 0, &c, nullptr, nullptr), SPEC_EINVAL);
    for (long long stride : {-1ll, (long long)INT64_MIN}) {
        spec_kv_cache d = c;
        d.token_stride = stride;
        EXPECT(spec_kv_append(fake, 256, 64, fake, 256, 64, fake, 128, 64, fake, 128, 64, SPEC_BF16, 1, 4, 2, 64, fi, fi,
                              static_cast<double*>(fake), 64, 1.0f, 0, &d, nullptr, nullptr), SPEC_EINVAL);
    }
    for (int pages : {-1, 0, most, 1 << 28}) {
        spec_kv_cache d = c;
        d.num_pages = pages;
        d.page_size = pages == most ? most : 16;
        EXPECT(spec_prefix_attention(fake, 256, 64, SPEC_BF16, 3, 4, &d, 1, fi, fi, 2, fi, fi, 3, fi, 1.0f,
                                     reinterpret_cast<void*>(0x2000), 256, 64, ff, fake, ~(size_t)0, nullptr), SPEC_EINVAL);
    }
    for (int max_pages : {-1, most})
        EXPECT(spec_prefix_attention(fake, 256, 64, SPEC_BF16, 3, 4, &c, 1, fi, fi, max_pages, fi, fi, 3, fi, 1.0f,
                                     reinterpret_cast<void*>(0x2000), 256, 64, ff, fake, ~(size_t)0, nullptr), SPEC_EINVAL);
    EXPECT(spec_tree_rows(fi, fi, fi, fi, 1, most, 1, fi, fi, fi, fi, nullptr), SPEC_EINVAL);
    EXPECT(spec_tree_rows(fi, fi, fi, fi, 1, 1, most, fi, fi, fi, fi, nullptr), SPEC_EINVAL);
    EXPECT(spec_verify_probs(fake, 1, 1, fake, 1, 1, SPEC_FP32, 1, 1, most, fi, nullptr, fake, fake, SPEC_FP32, 0, fi, fi,
                             nullptr, nullptr, nullptr, fake, ~(size_t)0, nullptr), SPEC_EINVAL);
    std::printf("%d checks, %d failures\n", checks, fails);
    return fails ? 1 : 0;
}
