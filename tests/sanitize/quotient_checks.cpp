// Every pair of mantissas of a 16-bit value x and of the largest value a of its
// block: x times the reciprocal of the block's factor, corrected once, is x / s
// rounded once. Built and run by tests/test_route_quotient.py.

#include <cmath>
#include <cstdio>
#include <initializer_list>

namespace {

float corrected_once(float x, float s, float inv) {
  const float q = x * inv;
  return std::fma(-std::fma(q, s, -x), inv, q);
}

}  // namespace

int main() {
  long pairs = 0, wrong = 0;
  const int mantissa_bits[] = {7, 10};  // BF16, FP16; an FP32 of either has no others
  const float largest[] = {448.0f, 57344.0f};
  for (int bits : mantissa_bits)
    for (float fmax : largest)
      for (int am = 0; am < 1 << bits; ++am)
        for (int xm = 0; xm < 1 << bits; ++xm)
          for (int sign = -1; sign <= 1; sign += 2)
            for (int e : {0, -40, 40}) {
              const float a = std::ldexp((float)((1 << bits) + am), e - bits), x = sign * std::ldexp((float)((1 << bits) + xm), e - bits);
              const float s = a / fmax, inv = 1.0f / s;
              ++pairs;
              if (corrected_once(x, s, inv) != x / s) ++wrong;
            }
  if (!std::signbit(corrected_once(-0.0f, 2.0f, 0.5f)) || std::signbit(corrected_once(0.0f, 2.0f, 0.5f))) ++wrong;
  std::printf("%ld pairs, %ld wrong\n", pairs, wrong);
  return wrong != 0;
}
