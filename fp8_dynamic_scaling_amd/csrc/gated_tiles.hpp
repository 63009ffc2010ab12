// gated_tiles.hpp -- which kernel takes a gated product, by its sizes. Host arithmetic alone, without HIP's headers.
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

namespace fp8dyn {

// The ping-pong kernel's shapes: two stages at least, and 32-bit offsets within a tile of A, in B and in the output.
inline bool gated_fast_eligible(int64_t F, int64_t K) {
  return K > 64 && 2 * F <= (1 << 22) && K <= (1 << 22) && 2 * F * K < ((int64_t)1 << 31);
}

constexpr int kGatedFew = 0, kGatedGeneric = -1;

// Rows of a workgroup's tile in the ping-pong kernel, or kGatedFew: the least of what each would take,
//   rounds over the CUs x (2 us + K x the time for 1024 of K),
// with times from measurements of one full round each (us for 1024 of K; the last with full precision):
//   k_gated_few, 64 rows x 16 features, two a CU         3.6
//   tiles of 64 x 128 features                           4.2 (8.2): a stage's loads bound it, not its products
//   tiles of 128 x 128 features                          6.8 (12.9)
//   tiles of 256 x 128 features, up to half of the CUs   9.6 (15.5); all of them 12.6 (22)
// Measured, k_gated_few / 64 / 128 / 256 rows, us: 256 x 2048 x 2048 11.9 / 12.6 / 15.0 / 23.1; 1024 x 1040 x 720
// 18.1 / 11.0 / 12.9 / 30.0; 1024 x 2048 x 2048 38.0 / 14.4 / 16.3 / 24.1; 256 x 14336 x 4096 124 / 53.9 / 43.4 /
// 51.3; 2048 x 4096 x 4096 269 / 100 / 69.5 / 56.5. An expert's rows are taken as the mean, and half a tile more.
// The times have no term for memory, and are too short where large weights bound a round (18.8 for 64 x 14336 x 4096).
// What the rule takes is the fastest there too, but for the last (k_gated_few / 64 / 128 rows, packed): 33 x 14336 x 4096
// 36.0 / 30.9 / 32.7; 64 x 14336 x 4096 39.2 / 35.8 / 37.9; 96 x 14336 x 4096 61.9 / 33.5 / 40.9; 64 x 8192 x 8192
// 37.2 / 58.9 / 60.1; 64 x 4096 x 4096 15.0 / 28.5 / 30.0; 64 x 14336 x 4096 row-major 39.8 / 43.7 / 46.1.
// Dense products that the ping-pong kernel does not take are k_gated_few's, which reads the weights once for each 64
// rows: 1024 x 66000 x 16400 12.9 ms, as a grouped product of one expert, kGatedGeneric, 5.7; 8192 x 14336 x 64 703 and
// 459 us.
// experts: 0 for a dense product. Grouped products that the ping-pong kernel does not take are kGatedGeneric.
inline int gated_tile_rows(int64_t M, int64_t F, int64_t K, int32_t experts, bool packed, bool exact, int cu_count) {
  const double cus = cu_count, k = (double)K / 1024.0;
  if (!experts && M <= 32) return kGatedFew;
  const double nt = (double)((F + 127) / 128);
  double best = 1e300;
  int rows = kGatedGeneric;
  if (!experts) {
    const double wgs = (double)((F + 15) / 16) * (double)((M + 63) / 64);
    best = std::ceil(wgs / (2.0 * cus)) * (2.0 + 3.6 * k);
    rows = kGatedFew;
  }
  if (packed || gated_fast_eligible(F, K)) {
    for (const int bm : {64, 128, 256}) {
      double mt = (double)((M + bm - 1) / bm);
      if (experts) {
        mt = (double)M / experts / bm + 0.5;
        mt = (mt < 1.0 ? 1.0 : mt) * experts;
      }
      const double tiles = mt * nt;
      const double c = bm == 64    ? (exact ? 8.2 : 4.2)
                       : bm == 128 ? (exact ? 12.9 : 6.8)
                       : 2.0 * tiles <= cus ? (exact ? 15.5 : 9.6)
                                            : (exact ? 22.0 : 12.6);
      const double t = std::ceil(tiles / cus) * (2.0 + c * k);
      if (t < best) best = t, rows = bm;
    }
  }
  return rows;
}

}  // namespace fp8dyn
