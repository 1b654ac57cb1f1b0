// Host check whether strided tensors share bytes. A tensor is n_t x n_h pieces of `width` adjacent
// bytes, piece (t, h) at base + t * s_t + h * s_h.
#pragma once
#include <algorithm>
#include <cstdint>

namespace ds4 {

using Wide = __int128;

struct Pieces {
  Wide base, s_t, s_h, low, high;  // low, high: the span, from the first byte to behind the last
  int64_t n_t, n_h, width;

  Pieces() = default;
  Pieces(const void* p, int64_t nt, int64_t st, int64_t nh, int64_t sh, int64_t w)
      : base(reinterpret_cast<uintptr_t>(p)), s_t(nt > 1 ? st : 0), s_h(nh > 1 ? sh : 0), n_t(nt),
        n_h(nh), width(w) {
    const Wide t = s_t * (n_t - 1), h = s_h * (n_h - 1);
    low = base + std::min<Wide>(0, t) + std::min<Wide>(0, h);
    high = base + std::max<Wide>(0, t) + std::max<Wide>(0, h) + width;
  }
};

// Whether some k in -(n - 1) .. n - 1 has low < c + k * step < high (n >= 1).
inline bool hits(Wide c, Wide step, int64_t n, Wide low, Wide high) {
  if (step < 0) step = -step;
  if (step == 0) return low < c && c < high;
  const Wide d = low - c;                       // the least k with k * step > d
  const Wide k = (d >= 0 ? d / step : -((-d + step - 1) / step)) + 1;
  const Wide last = n - 1, first = std::max(k, -last);
  return first <= last && c + first * step < high;
}

// Whether two pieces of one tensor share a byte.
inline bool overlaps_itself(const Pieces& a) {
  // the usual case: the longer stride steps over all of the shorter one's pieces
  const bool t_long = a.n_h < 2 || (a.n_t > 1 && a.s_t * a.s_t >= a.s_h * a.s_h);
  auto size = [](Wide s) { return s < 0 ? -s : s; };
  const Wide l = size(t_long ? a.s_t : a.s_h), s = size(t_long ? a.s_h : a.s_t);
  const int64_t n_l = t_long ? a.n_t : a.n_h, n_s = t_long ? a.n_h : a.n_t;
  const Wide inner = s * (n_s - 1) + a.width;
  if ((n_s < 2 || s >= a.width) && (n_l < 2 || l >= inner)) return false;
  // piece pairs (dt, dh) and (-dt, -dh) meet together: dh = 0 with dt >= 1, then dh >= 1
  if (a.n_t > 1 && size(a.s_t) < a.width) return true;
  for (int64_t dh = 1; dh < a.n_h; ++dh)
    if (hits(dh * a.s_h, a.s_t, a.n_t, -a.width, a.width)) return true;
  return false;
}

// Whether a piece of `a` and a piece of `b` (tensors of the same tokens) share a byte. Exact where
// the token strides agree or the spans are apart; spans that interleave at different token strides,
// or more than 2^20 pairs of heads at different head strides, count as shared.
inline bool overlap(const Pieces& a, const Pieces& b) {
  if (a.high <= b.low || b.high <= a.low) return false;
  if (a.s_t != b.s_t) return true;
  const Wide c = a.base - b.base, lo = -a.width, hi = b.width;
  // the heads of one token as one run from the first to the last
  const Wide low = std::min<Wide>(0, a.s_h * (a.n_h - 1)) - std::max<Wide>(0, b.s_h * (b.n_h - 1));
  const Wide high = std::max<Wide>(0, a.s_h * (a.n_h - 1)) - std::min<Wide>(0, b.s_h * (b.n_h - 1));
  if (!hits(c, a.s_t, a.n_t, lo - high, hi - low)) return false;
  if (a.n_h == 1 || b.n_h == 1 || a.s_h == b.s_h) {
    const Wide s = a.n_h == 1 ? b.s_h : a.s_h;
    for (int64_t dh = 1 - b.n_h; dh < a.n_h; ++dh)
      if (hits(c + dh * s, a.s_t, a.n_t, lo, hi)) return true;
    return false;
  }
  if (a.n_h * b.n_h > 1 << 20) return true;
  for (int64_t i = 0; i < a.n_h; ++i)
    for (int64_t j = 0; j < b.n_h; ++j)
      if (hits(c + i * a.s_h - j * b.s_h, a.s_t, a.n_t, lo, hi)) return true;
  return false;
}

// Whether `out` is `x` itself, written in place.
inline bool same(const Pieces& a, const Pieces& b) {
  return a.base == b.base && a.s_t == b.s_t && a.s_h == b.s_h && a.n_h == b.n_h && a.width == b.width;
}

}  // namespace ds4
