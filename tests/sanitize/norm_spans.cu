// The columns that the layer norm's kernels take for a segment, and the weights that its threads read, for column
// offsets that are not the widths': every start and end around a row, row length and vector width, on the host.  Prints
// "spans ok", or the first offsets that leave the row.
#include <climits>
#include <cstdio>
#include <initializer_list>

#include "norm_rows.cuh"

namespace {

template <int V, int L>
bool weights_inside(int col, int width, int cols) {
  for (int lane = 0; lane < L; ++lane) {
    const int first = lane * V < width ? col + lane * V : col;  // as the kernels pass it on
    for (int j = 0; j < tbe::kPer / V; ++j) {
      const bool in = (j * L + lane) * V < width;
      const int c = in ? first + j * L * V : first;
      if (c < 0 || c % V != 0 || c + V > cols) return false;
    }
  }
  return true;
}

template <int V>
bool check() {
  for (int cols : {V, 2 * V, 4 * V, 24 * V}) {
    for (int widest : {V, cols}) {
      auto one = [&](int c0, int c1) {
        int col, width;
        tbe::clamp_span<V>(c0, c1, cols, widest, &col, &width);
        const bool row = col >= 0 && width >= 0 && width <= widest && col % V == 0 && width % V == 0 && col + width <= cols;
        if (row && weights_inside<V, 4>(col, width, cols) && weights_inside<V, 32>(col, width, cols)) return true;
        std::printf("vectors of %d, %d columns, offsets %d and %d: column %d, width %d\n", V, cols, c0, c1, col, width);
        return false;
      };
      for (int c0 = -V - 1; c0 <= cols + V + 1; ++c0)
        for (int c1 = -V - 1; c1 <= cols + V + 1; ++c1)
          if (!one(c0, c1)) return false;
      for (int c0 : {INT_MIN, -1, 0, cols, INT_MAX})
        for (int c1 : {INT_MIN, -1, 0, cols, INT_MAX})
          if (!one(c0, c1)) return false;
      // offsets that agree are taken as they are
      for (int c0 = 0; c0 < cols; c0 += V)
        for (int w = V; w <= widest && c0 + w <= cols; w += V) {
          int col, width;
          tbe::clamp_span<V>(c0, c0 + w, cols, widest, &col, &width);
          if (col != c0 || width != w) return false;
        }
    }
  }
  return true;
}

}  // namespace

int main() {
  if (!check<1>() || !check<4>() || !check<8>()) return 1;
  std::puts("spans ok");
  return 0;
}
