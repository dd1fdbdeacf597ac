// Host check of the paged cache's index arithmetic and scale exponents (no
// GPU, no library): the row coordinate of every 32-token tile lies inside its
// page's head, a page that is not there gives the row one past the last, and
// the exponent is the smallest that holds amax within 448 * 2^e.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "gdn_kv.cuh"

int main() {
    long checks = 0;
    for (int lp = 5; lp <= 7; ++lp)
        for (int Hkv : {1, 3, 8})
            for (int pages : {1, 7, 65536, (int)(0x7fffff00LL / (Hkv << lp))})
                for (int page : {-2147483647 - 1, -1, 0, 1, pages / 2, pages - 1, pages, pages + 1, 2147483647})
                    for (int h = 0; h < Hkv; ++h)
                        for (int pos : {0, 32, 96, 4096 + 64, 2147483616}) {
                            const long long rows = (long long)pages * Hkv << lp;
                            const long long y = gdn::cache_row(page, pages, Hkv, h, lp, pos);
                            const bool there = page >= 0 && page < pages;
                            const long long first = there ? ((long long)page * Hkv + h) << lp : rows;
                            const long long want = there ? first + pos % (1 << lp) : rows;
                            if (y != want || y < 0 || (there && y + 32 > rows)) {
                                printf("row of page %d head %d pos %d: %lld, want %lld of %lld\n", page, h, pos, y, want, rows);
                                return 1;
                            }
                            ++checks;
                        }
    for (unsigned bits = 0; bits < 0x7f80u; ++bits) {  // every finite bf16 magnitude
        const unsigned w = bits << 16;
        float x;
        memcpy(&x, &w, 4);
        const int e = gdn::scale_exp_of_bf16(bits);
        const bool holds = (double)x <= std::ldexp(448.0, e), least = e == gdn::kScaleMinExp || (double)x > std::ldexp(448.0, e - 1);
        if (e < gdn::kScaleMinExp || e > gdn::kScaleMaxExp || !holds || !least) {
            printf("exponent of %g: %d\n", x, e);
            return 1;
        }
        ++checks;
    }
    printf("%ld indices and exponents OK\n", checks);
    return 0;
}
