// binding.cu -- calls with packed arguments (a4w4_binding.h).
#include <cstdint>
#include <cstring>

#include "a4w4.h"
#include "a4w4_binding.h"

namespace {

template <int N>
struct Words {
  int64_t w[N];
  explicit Words(const void* packed) { std::memcpy(w, packed, sizeof(w)); }
  template <typename T>
  T* ptr(int i) const { return reinterpret_cast<T*>(static_cast<uintptr_t>(w[i])); }
  void* any(int i) const { return ptr<void>(i); }
  int num(int i) const { return static_cast<int>(w[i]); }
  float real(int i) const {
    double d;
    std::memcpy(&d, &w[i], sizeof(d));
    return static_cast<float>(d);
  }
};

}  // namespace

extern "C" {

int a4w4_packed_gemm_w8a8(const void* packed) {
  if (packed == nullptr) return A4W4_ERR_ARG;
  const Words<11> a(packed);
  return a4w4_gemm_w8a8(a.any(0), a.num(1), a.num(2), a.any(3), a.ptr<const float>(4), a.num(5), a.any(6), a.any(7),
                        static_cast<size_t>(a.w[8]), static_cast<unsigned int>(a.w[9]), a.any(10));
}

int a4w4_packed_kv_read(const void* packed) {
  if (packed == nullptr) return A4W4_ERR_ARG;
  const Words<10> a(packed);
  return a4w4_kv_read(a.any(0), a.num(1), a.num(2), a.ptr<const int32_t>(3), a.num(4), a.num(5), a.num(6), a.any(7),
                      a.any(8), a.any(9));
}

int a4w4_packed_moe_route(const void* packed) {
  if (packed == nullptr) return A4W4_ERR_ARG;
  const Words<17> a(packed);
  return a4w4_moe_route(a.any(0), a.num(1), a.w[2], a.ptr<const int32_t>(3), a.num(4), a.num(5), a.num(6),
                        a.ptr<const float>(7), a.num(8), a.num(9), a.num(10), a.num(11), a.num(12), a.real(13),
                        a.ptr<int32_t>(14), a.ptr<float>(15), a.any(16));
}

int a4w4_packed_qk_norm_rope(const void* packed) {
  if (packed == nullptr) return A4W4_ERR_ARG;
  const Words<20> a(packed);
  return a4w4_qk_norm_rope(a.any(0), a.w[1], a.any(2), a.w[3], a.ptr<const int32_t>(4), a.num(5), a.num(6), a.num(7),
                           a.num(8), a.ptr<const float>(9), a.ptr<const float>(10), a.real(11), a.ptr<const float>(12),
                           a.num(13), a.num(14), a.any(15), a.w[16], a.any(17), a.w[18], a.any(19));
}

int a4w4_packed_kv_append_rope(const void* packed) {
  if (packed == nullptr) return A4W4_ERR_ARG;
  const Words<24> a(packed);
  return a4w4_kv_append_rope(a.any(0), a.w[1], a.any(2), a.w[3], a.any(4), a.w[5], a.ptr<const int32_t>(6),
                             a.ptr<const int32_t>(7), a.num(8), a.num(9), a.num(10), a.num(11), a.ptr<const float>(12),
                             a.ptr<const float>(13), a.real(14), a.ptr<const float>(15), a.num(16), a.num(17), a.any(18),
                             a.w[19], a.any(20), a.num(21), a.num(22), a.any(23));
}

}  // extern "C"
