// Walks the addresses that the 4-bit product's copies of activations read, on the
// host: every copy of every lane, step and tile, for every count of rows in a block.
// As the hardware does, an offset is within the buffer when it is below the
// buffer's size less the wave's base, both unsigned: the base must not pass the
// size, the chunks of the block's rows below K must be read from where they are,
// and nothing else may be read.
#include <stdio.h>

#include "gemm_w4.hpp"

template <int XR>
static long walk(int K) {
  using Tile = mmk::W4Tile<XR>;
  const int kblocks = (K + 127) / 128;
  const uint32_t row_bytes = 2u * (uint32_t)K;
  long bad = 0;
  for (int have = 1; have <= XR; ++have) {
    const uint32_t size = (uint32_t)have * row_bytes;
    for (int kb = 0; kb < kblocks; ++kb)
      for (int half = 0; half < (Tile::kHalves ? 2 : 1); ++half) {
        const bool last = kb == kblocks - 1;
        const uint32_t base = Tile::base(kb, half, last);
        bad += base > size;
        for (int i = 0; i < Tile::kCopies; ++i)
          for (int lane = 0; lane < 64; ++lane) {
            const uint32_t off =
                Tile::offset(i, lane, row_bytes) + (last ? Tile::tail(Tile::kHalves ? half : i & 3, lane, K) : 0u);
            const int row = Tile::row(i, lane), k = 128 * kb + (Tile::kHalves ? 64 * half : 0) + 8 * Tile::chunk(i, lane);
            const bool want = row < have && k < K, got = off < size - base;
            bad += want != got || (want && off + base != (uint32_t)row * row_bytes + 2u * (uint32_t)k);
          }
      }
  }
  if (bad) printf("%d rows, K = %d: %ld\n", XR, K, bad);
  return bad;
}

int main() {
  long bad = 0;
  for (int K = 8; K <= 424; K += 8)
    bad += walk<4>(K) + walk<16>(K) + walk<32>(K) + walk<48>(K) + walk<64>(K);
  for (int K : {4104, 1 << 22}) {
    // (K is large: the last blocks of rows and steps only matter through 32-bit offsets)
    const uint32_t row_bytes = 2u * (uint32_t)K;
    bad += mmk::W4Tile<64>::offset(7, 63, row_bytes) + mmk::W4Tile<64>::base((K + 127) / 128 - 1, 1, true) >= 1u << 31;
  }
  return bad != 0;
}
