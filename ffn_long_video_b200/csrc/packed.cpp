// The generation calls with their arguments packed into 8-byte words (integers,
// pointers and doubles in the order of the C prototypes), for a caller to whom
// every argument of a foreign call costs time: the Python binding converts one
// pointer instead of some forty arguments (4.7 -> 1.1 us per call on the host).
// The words carry what the prototypes take, nothing is added or left out.
#include <cstring>

#include "adaspark.h"

namespace {

struct Words {
  const unsigned char* at;
  int64_t i() {
    int64_t v;
    std::memcpy(&v, at, 8);
    at += 8;
    return v;
  }
  int n() {  // a number outside int becomes one that every call refuses
    const int64_t v = i();
    return v == (int)v ? (int)v : INT32_MIN;
  }
  double f() {
    double v;
    std::memcpy(&v, at, 8);
    at += 8;
    return v;
  }
  template <typename T>
  T* p() {
    return reinterpret_cast<T*>(i());
  }
};

}  // namespace

extern "C" {

int adaspark_packed_qk_rope(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const void* Q = w.p<const void>(); const int64_t q_ts = w.i(), q_hs = w.i();
  const void* K = w.p<const void>(); const int64_t k_ts = w.i(), k_hs = w.i();
  const int dtype = w.n();
  const int32_t* pos = w.p<const int32_t>(); const int axes = w.n();
  const int32_t sec[3] = {w.n(), w.n(), w.n()};
  const double* freq = w.p<const double>(); const int rot = w.n(), il = w.n();
  const float mag = (float)w.f();
  const void *wq = w.p<const void>(), *wk = w.p<const void>();
  const float eps = (float)w.f();
  const int n = w.n(), hq = w.n(), hkv = w.n(), d = w.n();
  void* Qo = w.p<void>(); const int64_t qo_ts = w.i(), qo_hs = w.i();
  void* Ko = w.p<void>(); const int64_t ko_ts = w.i(), ko_hs = w.i();
  void* stream = w.p<void>();
  return adaspark_qk_rope(Q, q_ts, q_hs, K, k_ts, k_hs, dtype, pos, axes, sec, freq, rot, il, mag,
                          wq, wk, eps, n, hq, hkv, d, Qo, qo_ts, qo_hs, Ko, ko_ts, ko_hs, stream);
}

int adaspark_packed_qk_rope_append(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const void* Q = w.p<const void>(); const int64_t q_ts = w.i(), q_hs = w.i();
  const void* K = w.p<const void>(); const int64_t k_ts = w.i(), k_hs = w.i();
  const void* V = w.p<const void>(); const int64_t v_ts = w.i(), v_hs = w.i();
  const int dtype = w.n();
  const int32_t* pos = w.p<const int32_t>(); const int axes = w.n();
  const int32_t sec[3] = {w.n(), w.n(), w.n()};
  const double* freq = w.p<const double>(); const int rot = w.n(), il = w.n();
  const float mag = (float)w.f();
  const void *wq = w.p<const void>(), *wk = w.p<const void>();
  const float eps = (float)w.f();
  const int n = w.n(), hq = w.n(), hkv = w.n(), d = w.n();
  const int32_t* slots = w.p<const int32_t>();
  void *kc = w.p<void>(), *vc = w.p<void>();
  const int64_t c_ps = w.i(), c_ts = w.i(), c_hs = w.i();
  const int pages = w.n(), page = w.n();
  void* Qo = w.p<void>(); const int64_t qo_ts = w.i(), qo_hs = w.i();
  void* stream = w.p<void>();
  return adaspark_qk_rope_append(Q, q_ts, q_hs, K, k_ts, k_hs, V, v_ts, v_hs, dtype, pos, axes, sec,
                                 freq, rot, il, mag, wq, wk, eps, n, hq, hkv, d, slots, kc, vc,
                                 c_ps, c_ts, c_hs, pages, page, Qo, qo_ts, qo_hs, stream);
}

int adaspark_packed_kv_append(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const void* K = w.p<const void>(); const int64_t k_ts = w.i(), k_hs = w.i();
  const void* V = w.p<const void>(); const int64_t v_ts = w.i(), v_hs = w.i();
  const int dtype = w.n(), n = w.n(), hkv = w.n(), d = w.n();
  const int32_t* slots = w.p<const int32_t>();
  void *kc = w.p<void>(), *vc = w.p<void>();
  const int64_t c_ps = w.i(), c_ts = w.i(), c_hs = w.i();
  const int pages = w.n(), page = w.n();
  void* stream = w.p<void>();
  return adaspark_kv_append(K, k_ts, k_hs, V, v_ts, v_hs, dtype, n, hkv, d, slots, kc, vc, c_ps,
                            c_ts, c_hs, pages, page, stream);
}

int adaspark_packed_qk_rope_backward(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const void* gQ = w.p<const void>(); const int64_t gq_ts = w.i(), gq_hs = w.i();
  const void* gK = w.p<const void>(); const int64_t gk_ts = w.i(), gk_hs = w.i();
  const int dy = w.n();
  const void* Q = w.p<const void>(); const int64_t q_ts = w.i(), q_hs = w.i();
  const void* K = w.p<const void>(); const int64_t k_ts = w.i(), k_hs = w.i();
  const int dtype = w.n();
  const int32_t* pos = w.p<const int32_t>(); const int axes = w.n();
  const int32_t sec[3] = {w.n(), w.n(), w.n()};
  const double* freq = w.p<const double>(); const int rot = w.n(), il = w.n();
  const float mag = (float)w.f();
  const void *wq = w.p<const void>(), *wk = w.p<const void>();
  const float eps = (float)w.f();
  const int n = w.n(), hq = w.n(), hkv = w.n(), d = w.n();
  float *dQ = w.p<float>(), *dK = w.p<float>(), *dwq = w.p<float>(), *dwk = w.p<float>();
  void* ws = w.p<void>(); const int64_t bytes = w.i();
  void* stream = w.p<void>();
  return adaspark_qk_rope_backward(gQ, gq_ts, gq_hs, gK, gk_ts, gk_hs, dy, Q, q_ts, q_hs, K, k_ts,
                                   k_hs, dtype, pos, axes, sec, freq, rot, il, mag, wq, wk, eps, n,
                                   hq, hkv, d, dQ, dK, dwq, dwk, ws, (size_t)bytes, stream);
}

int adaspark_packed_kv_plan(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const int32_t *old_lens = w.p<const int32_t>(), *new_lens = w.p<const int32_t>();
  const int n_seqs = w.n(), page = w.n();
  int32_t* table = w.p<int32_t>(); const int64_t stride = w.i(); const int cols = w.n();
  int32_t* free_pages = w.p<int32_t>(); const int n_pages = w.n();
  int32_t *n_free = w.p<int32_t>(), *starts = w.p<int32_t>(), *slots = w.p<int32_t>(),
          *pos = w.p<int32_t>();
  const int rows = w.n();
  void* ws = w.p<void>(); const int64_t bytes = w.i();
  void* stream = w.p<void>();
  return adaspark_kv_plan(old_lens, new_lens, n_seqs, page, table, stride, cols, free_pages,
                          n_pages, n_free, starts, slots, pos, rows, ws, (size_t)bytes, stream);
}

int adaspark_packed_decode_attn(const void* words) {
  Words w{static_cast<const unsigned char*>(words)};
  const void* Q = w.p<const void>(); const int64_t q_ts = w.i(), q_hs = w.i();
  const void *kc = w.p<const void>(), *vc = w.p<const void>();
  const int64_t c_ps = w.i(), c_ts = w.i(), c_hs = w.i();
  const int pages = w.n(), page = w.n(), dtype = w.n();
  const int32_t* table = w.p<const int32_t>(); const int64_t stride = w.i(); const int cols = w.n();
  const int32_t* lens = w.p<const int32_t>();
  const int n = w.n(), hq = w.n(), hkv = w.n(), d = w.n();
  const float scale = (float)w.f();
  void* out = w.p<void>(); float* lse = w.p<float>();
  void* ws = w.p<void>(); const int64_t bytes = w.i();
  void* stream = w.p<void>();
  return adaspark_decode_attn(Q, q_ts, q_hs, kc, vc, c_ps, c_ts, c_hs, pages, page, dtype, table,
                              stride, cols, lens, n, hq, hkv, d, scale, out, lse, ws,
                              (size_t)bytes, stream);
}

}  // extern "C"
