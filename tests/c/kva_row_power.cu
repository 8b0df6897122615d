// Host check of the power of two that brings a query row into fp16's range: for
// every largest value, the way back undoes it.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "kva_attention.cuh"

using namespace kvw;

static float number(uint32_t bits) {
    float f;
    std::memcpy(&f, &bits, 4);
    return f;
}

int main() {
    long checks = 0;
    for (uint32_t top = 0; top < 0x8000u; ++top) {
        uint32_t u, d;
        row_exponents(top, u, d);
        const double up = number(u << 23), down = number(d << 23), x = number(top << 16);
        bool ok = u >= 1 && u <= 254 && d >= 1 && d <= 254 && up * down == 1.0;
        if (top == 0 || (top >> 7) == 255)
            ok &= up == 1.0;
        else if (x >= std::ldexp(1.0, -112))
            ok &= x * up >= std::ldexp(1.0, 14) && x * up < std::ldexp(1.0, 15);
        else  // a multiple of fp16's smallest step, below its largest number
            ok &= x * up < std::ldexp(1.0, 14) && std::fmod(x * up, std::ldexp(1.0, -24)) == 0.0;
        if (!ok) {
            printf("top %04x: up %g, down %g\n", top, up, down);
            return 1;
        }
        ++checks;
    }
    printf("%ld checks, 0 mismatches\n", checks);
    return 0;
}
