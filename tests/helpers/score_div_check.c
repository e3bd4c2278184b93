/* Checks, in IEEE binary32 with fused multiply-add, the two divisions of the routing scores.  Prints "checked bad" for
 *   1. the reciprocal r + r (1 - x r) from the start r = RN(1 / x), every x in [1, 2);
 *   2. the same from starts an ulp below and above;
 *   3. the quotient q + r (a - q b), q = RN(a r), r = RN(1 / b), at the a next to a rounding midpoint: for every odd
 *      and argv 1-th even significand b, the a with a 2^k = (2 n + 1) b + d for every |d| <= argv 2 (found by the
 *      inverse of b modulo 2^k), where the rounding is decided by the least margin;
 *   4. argv 3 random pairs. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

static float u2f(uint32_t u) { float f; memcpy(&f, &u, 4); return f; }
static uint32_t f2u(float f) { uint32_t u; memcpy(&u, &f, 4); return u; }
static float step(float x, float r) { return fmaf(fmaf(-x, r, 1.0f), r, r); }
static int wrong(float a, float b) {
  volatile float one = 1.0f, want = a / b;
  const float r = one / b;
  volatile float q = a * r; /* a separate multiply */
  return fmaf(fmaf(-q, b, a), r, q) != want;
}

static uint64_t st = 0x9E3779B97F4A7C15ull;
static uint32_t rnd(void) { /* xorshift64* */
  st ^= st >> 12; st ^= st << 25; st ^= st >> 27;
  return (uint32_t)((st * 0x2545F4914F6CDD1Dull) >> 32);
}

int main(int argc, char **argv) {
  if (argc < 4) return 2;
  const int every = atoi(argv[1]), most = atoi(argv[2]);
  const long pairs = atol(argv[3]);
  long n = 0, bad[3] = {0, 0, 0};
  for (uint32_t m = 0; m < 1u << 23; ++m, ++n) {
    volatile float one = 1.0f;
    const float x = u2f(0x3F800000u | m), t = one / x;
    for (int d = -1; d <= 1; ++d) bad[d + 1] += step(x, u2f(f2u(t) + d)) != t;
  }
  printf("%ld %ld\n%ld %ld\n", n, bad[1], 2 * n, bad[0] + bad[2]);
  long checked = 0, missed = 0;
  for (uint64_t b = 1u << 23; b < 1u << 24; ++b) {
    if (b % 2 == 0 && (b / 2) % (uint64_t)every != 0) continue;
    const int twos = __builtin_ctzll(b);
    const uint64_t odd = b >> twos;
    uint64_t inv = odd; /* modulo 2^64, by Newton's steps */
    for (int i = 0; i < 6; ++i) inv *= 2 - odd * inv;
    for (int k = 24; k <= 25; ++k) { /* quotients in [1, 2) and [1/2, 1) */
      for (int64_t d = -most; d <= most; ++d) {
        /* (2 n + 1) odd = -d modulo 2^(k - twos), d in units of 2^twos */
        const uint64_t mod = k - twos, mask = ((uint64_t)1 << mod) - 1;
        if (d % 2 == 0) continue;
        for (uint64_t top = 0; top < ((uint64_t)1 << twos) && top < 4; ++top) {
          const uint64_t mid = (((uint64_t)(-d) * inv) & mask) + (top << mod); /* 2 n + 1, 25 bits */
          if (mid < (1u << 24) || mid >= (1u << 25)) continue;
          const uint64_t num = mid * b + (uint64_t)(d << twos);
          const uint64_t a = num >> k;
          if (num & (((uint64_t)1 << k) - 1) || a < (1u << 23) || a >= (1u << 24)) continue;
          ++checked;
          missed += wrong((float)a, (float)b);
        }
      }
    }
  }
  printf("%ld %ld\n", checked, missed);
  missed = 0;
  for (long i = 0; i < pairs; ++i)
    missed += wrong(u2f(0x3F800000u | (rnd() & 0x7FFFFF)), u2f(0x3F800000u | (rnd() & 0x7FFFFF)));
  printf("%ld %ld\n", pairs, missed);
  return 0;
}
