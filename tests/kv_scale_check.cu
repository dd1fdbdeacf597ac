// Host check of a block's marked scale (no GPU, no library): always a NaN, it gives the
// scale back to the rows before the first one that is not finite, and to no others.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "gdn_kv.cuh"

static uint32_t bits_of(float x) {
    uint32_t w;
    memcpy(&w, &x, 4);
    return w;
}
static float float_of(uint32_t w) {
    float x;
    memcpy(&x, &w, 4);
    return x;
}

int main() {
    long checks = 0;
    for (int e = -126; e <= 127; ++e)
        for (int row = 0; row < 128; ++row) {
            const uint32_t scale = bits_of(std::ldexp(1.0f, e)), marked = gdn::marked_scale(scale, row);
            if (!std::isnan(float_of(marked))) return printf("2^%d row %d: %08x is a number\n", e, row, marked), 1;
            for (int at = 0; at <= 128; ++at, ++checks) {
                const uint32_t got = gdn::scale_before(marked, at), want = at <= row ? scale : marked;
                if (got != want) return printf("2^%d row %d at %d: %08x, want %08x\n", e, row, at, got, want), 1;
            }
        }
    // numbers, and NaNs that are no marks, come back as they are
    for (float x : {0.0f, -1.0f, 1.5f, 3e38f, 1e-40f, INFINITY, -INFINITY, 0.0009765625f})
        for (int at : {0, 1, 127, 128}) {
            if (gdn::scale_before(bits_of(x), at) != bits_of(x)) return printf("%g changed\n", x), 1;
            ++checks;
        }
    for (uint32_t w : {0x7fffffffu, 0x7fc00000u, 0xffc08000u, 0x7f808001u, 0xffffffffu, 0x7fc08000u, 0x7fc080ffu, 0x7fd08080u})
        for (int at : {0, 1, 127, 128}) {
            if (!std::isnan(float_of(gdn::scale_before(w, at)))) return printf("%08x at %d is a number\n", w, at), 1;
            ++checks;
        }
    // scales that are no powers of two are lost
    for (float x : {0.0f, -2.0f, 1.5f, 3e38f, 1e-40f, INFINITY, NAN})
        if (gdn::marked_scale(bits_of(x), 5) != gdn::kLostScale) return printf("%g is kept\n", x), 1;
    printf("%ld scales OK\n", checks);
    return 0;
}
