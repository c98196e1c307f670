// Order of an expert's output tiles in bands of its row tiles (host and device).
#pragma once

namespace mfsdp {

struct BandTile {
  int ti, tj;     // row tile, column tile
};

// Tile number `local` of rows x nq, band by band, columns in order within one: as many
// bands as are nearest to `band` row tiles each, of heights that differ by at most
// one, the higher ones first.
constexpr BandTile band_tile(int rows, int nq, int band, int local) {
  const int bands = rows < band ? 1 : (rows + band / 2) / band;
  const int low = rows / bands, higher = rows % bands;
  const int lows = higher * (low + 1);          // first row tile of the lower bands
  const bool in_low = local >= lows * nq;
  const int height = in_low ? low : low + 1, at = in_low ? local - lows * nq : local;
  const int b = at / (height * nq), r = at - b * (height * nq);
  return {(in_low ? lows : 0) + b * height + r % height, r / height};
}

}  // namespace mfsdp
