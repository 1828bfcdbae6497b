// The quotient that the state cache's codes are taken from lies on the same side of every border between two
// codes as the exact x / s, and is a number: for values on and beside the borders of scales of every
// size, and for values far below their scale.  Host arithmetic only; long double holds border x scale.
#include <math.h>
#include <stdio.h>

#include <vector>

#include "kda_state_cache.hpp"

static std::vector<float> borders(bool f8) {
    std::vector<float> b;
    if (!f8) {
        for (int i = 0; i < 127; ++i) b.push_back(i + 0.5f);
        return b;
    }
    std::vector<float> v;  // e4m3: subnormals, then 8 values an exponent up to 448
    for (int i = 0; i < 8; ++i) v.push_back(ldexpf((float)i, -9));
    for (int e = -6; e <= 8; ++e)
        for (int i = 8; i < 16; ++i)
            if (ldexpf((float)i, e - 3) <= 448.f) v.push_back(ldexpf((float)i, e - 3));
    for (size_t i = 0; i + 1 < v.size(); ++i) b.push_back((v[i] + v[i + 1]) / 2);
    return b;
}

static int sign(long double v) { return v > 0 ? 1 : v < 0 ? -1 : 0; }

static long checked = 0;
static int check(float x, float s, const std::vector<float>& all) {
    for (int neg = 0; neg < 2; ++neg) {
        const float v = neg ? -x : x, q = kda::beside_border(v, s);
        ++checked;
        if (!isfinite(q) || fabsf(q) > 1000.f) {
            printf("%a / %a gives %a\n", v, s, q);
            return 1;
        }
        for (float m : all)
            for (int side = -1; side <= 1; side += 2)
                if (sign((long double)q - side * m) != sign((long double)v - (long double)(side * m) * s)) {
                    printf("%a / %a gives %a, on the wrong side of %a\n", v, s, q, side * m);
                    return 1;
                }
    }
    return 0;
}

int main() {
    const std::vector<float> i8 = borders(false), f8 = borders(true);
    // the least scales, those around the least normal number, and ordinary ones
    const float scales[] = {0x1p-149f, 0x1.8p-148f, 0x1p-140f, 0x1.fffffcp-127f, 0x1p-126f, 0x1.000002p-126f, 0x1.aaaaaap-126f,
                            0x1.23456p-125f, 0x1.fffffep-124f, 0x1.555556p-120f, 0x1.fffffep-61f, 0x1.000002p-60f, 0.7f, 1.f, 1.1f, 777.7f,
                            2.23f, 2.2e7f, 3.3e-5f, 1.9e30f, 2.3e-30f, 7e35f};
    int bad = 0;
    for (float s : scales) {
        for (const auto* b : {&i8, &f8})
            for (float m : *b) {
                float x = (float)((long double)m * s);
                for (int k = 0; k < 3; ++k) x = nextafterf(x, 0.f);
                for (int k = 0; k < 7; ++k, x = nextafterf(x, INFINITY)) bad += check(x, s, *b);
            }
        for (float x = 0x1p-149f; x < s; x *= 3.f) bad += check(x, s, i8) + check(x, s, f8);
        bad += check(0.f, s, i8) + check(0.f, s, f8);
        if (bad) break;
    }
    if (!bad) printf("state codes check ok: %ld quotients\n", checked);
    return bad != 0;
}
