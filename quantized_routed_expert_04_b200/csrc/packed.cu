// The calls of the norm and of router training with their arguments in one
// array of 8-byte words, for the Python binding: a foreign-function call that
// converts 12 to 18 arguments one by one takes about as long as a kernel launch
// (1.5 us for 17), one that passes an array 0.4 us.  Word for word the arguments
// of the functions in include/strata_moe.h, in their order, the stream last;
// floats as doubles.  Not part of the C interface.
#include <string.h>

#include "strata_moe.h"

namespace {

struct Words {
  const int64_t *w;
  template <typename T>
  T *ptr() { return reinterpret_cast<T *>(*w++); }
  long long num() { return *w++; }
  // an int argument: what does not fit is refused as any negative number is
  int integer() {
    const long long v = *w++;
    return v < -1 || v > 2147483647LL ? -1 : (int)v;
  }
  float real() {
    double d;
    memcpy(&d, w++, sizeof d);
    return (float)d;
  }
  strata_stream_t stream() { return reinterpret_cast<strata_stream_t>(*w++); }
};

}  // namespace

// (an initialiser list is evaluated from left to right, a call's arguments are
// not: every word is read into a variable first)
extern "C" {

strata_status strata_packed_rmsnorm(const int64_t *words) {
  Words a{words};
  const int dtype = a.integer();
  const auto x = a.ptr<const void>();
  const long long ldx = a.num();
  const auto r = a.ptr<const void>();
  const long long ldr = a.num();
  const auto weight = a.ptr<const float>();
  const float eps = a.real();
  const int T = a.integer(), H = a.integer();
  const auto ro = a.ptr<void>();
  const long long ldro = a.num();
  const auto out = a.ptr<void>();
  const long long ldo = a.num();
  const auto q8 = a.ptr<void>();
  const auto scales = a.ptr<float>();
  const int group = a.integer();
  return strata_rmsnorm(dtype, x, ldx, r, ldr, weight, eps, T, H, ro, ldro, out, ldo, q8, scales,
                        group, a.stream());
}

strata_status strata_packed_rmsnorm_backward(const int64_t *words) {
  Words a{words};
  const int dtype = a.integer();
  const auto h = a.ptr<const void>();
  const long long ldh = a.num();
  const auto weight = a.ptr<const float>();
  const float eps = a.real();
  const auto dout = a.ptr<const void>();
  const long long lddo = a.num();
  const auto dsum = a.ptr<const void>();
  const long long ldds = a.num();
  const int T = a.integer(), H = a.integer();
  const auto dx = a.ptr<void>();
  const long long lddx = a.num();
  const auto dweight = a.ptr<float>();
  const auto ws = a.ptr<void>();
  const size_t ws_bytes = (size_t)a.num();
  return strata_rmsnorm_backward(dtype, h, ldh, weight, eps, dout, lddo, dsum, ldds, T, H, dx, lddx,
                                 dweight, ws, ws_bytes, a.stream());
}

strata_status strata_packed_balance(const int64_t *words) {
  Words a{words};
  const auto h = a.ptr<strata_moe>();
  const auto logits = a.ptr<const float>();
  const auto idx = a.ptr<const int32_t>();
  const int T = a.integer();
  const auto seq_off = a.ptr<const int32_t>();
  const int n_seq = a.integer();
  const auto mask = a.ptr<const uint8_t>();
  const float coef = a.real();
  const auto counts = a.ptr<int32_t>(), tokens = a.ptr<int32_t>();
  const auto loss = a.ptr<float>();
  const auto ws = a.ptr<void>();
  const size_t ws_bytes = (size_t)a.num();
  return strata_moe_balance(h, logits, idx, T, seq_off, n_seq, mask, coef, counts, tokens, loss, ws,
                            ws_bytes, a.stream());
}

strata_status strata_packed_balance_backward(const int64_t *words) {
  Words a{words};
  const auto h = a.ptr<strata_moe>();
  const auto logits = a.ptr<const float>();
  const int T = a.integer();
  const auto seq_off = a.ptr<const int32_t>();
  const int n_seq = a.integer();
  const auto mask = a.ptr<const uint8_t>();
  const float coef = a.real();
  const auto counts = a.ptr<const int32_t>(), tokens = a.ptr<const int32_t>();
  const auto dloss = a.ptr<const float>();
  const auto dlogits = a.ptr<float>();
  return strata_moe_balance_backward(h, logits, T, seq_off, n_seq, mask, coef, counts, tokens, dloss,
                                     dlogits, a.stream());
}

strata_status strata_packed_route_backward(const int64_t *words) {
  Words a{words};
  const auto h = a.ptr<strata_moe>();
  const auto x = a.ptr<const void>();
  const int T = a.integer();
  const auto logits = a.ptr<const float>();
  const auto idx = a.ptr<const int32_t>();
  const auto dw = a.ptr<const float>(), dlogits = a.ptr<const float>();
  const auto dW = a.ptr<float>(), db = a.ptr<float>();
  const auto dx = a.ptr<void>();
  const auto ws = a.ptr<void>();
  const size_t ws_bytes = (size_t)a.num();
  return strata_moe_route_backward(h, x, T, logits, idx, dw, dlogits, dW, db, dx, ws, ws_bytes,
                                   a.stream());
}

}  // extern "C"
