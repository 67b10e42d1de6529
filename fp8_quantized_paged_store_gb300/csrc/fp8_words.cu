// fp8_words.cu — the operators on the paged E4M3 cache, called with their
// arguments as an array of 64-bit words. For bindings that convert arguments
// one by one: through ctypes an append with its 40 took 23 us of host time,
// and 18 us with one array.
#include <cstdint>

#include "kvq_fp8.h"

namespace {

template <typename T>
T* ptr(int64_t w) {
  return reinterpret_cast<T*>(static_cast<uintptr_t>(w));
}

// A 32-bit argument; one that does not fit becomes a value that the functions
// refuse.
int32_t i32(int64_t w) { return w < -1 || w > INT32_MAX ? -1 : static_cast<int32_t>(w); }

}  // namespace

extern "C" int add_rmsnorm_fp8_words(const int64_t* w, int64_t count, float eps,
                                     cudaStream_t stream) {
  if (!w || count != 15) return KVQ_EINVAL;
  return add_rmsnorm_fp8(ptr<void>(w[0]), w[1], ptr<void>(w[2]), w[3], ptr<void>(w[4]), eps,
                         i32(w[5]), w[6], w[7], i32(w[8]), ptr<uint8_t>(w[9]), w[10],
                         ptr<float>(w[11]), w[12], ptr<void>(w[13]), w[14], stream);
}

extern "C" int rope_fp8_kv_append_words(const int64_t* w, int64_t count, cudaStream_t stream) {
  if (!w || count != 39) return KVQ_EINVAL;
  return rope_fp8_kv_append(
      ptr<void>(w[0]), w[1], w[2], ptr<void>(w[3]), w[4], w[5], ptr<void>(w[6]), w[7], w[8],
      ptr<void>(w[9]), w[10], w[11], i32(w[12]), w[13], w[14], w[15], w[16], ptr<float>(w[17]),
      w[18], w[19], w[20], i32(w[21]), ptr<int64_t>(w[22]), ptr<uint8_t>(w[23]),
      ptr<uint8_t>(w[24]), w[25], w[26], w[27], w[28], w[29], ptr<uint8_t>(w[30]),
      ptr<uint8_t>(w[31]), w[32], ptr<int64_t>(w[33]), w[34], w[35], ptr<int64_t>(w[36]),
      ptr<int64_t>(w[37]), w[38], stream);
}

extern "C" int fp8_paged_attention_words(const int64_t* w, int64_t count, float sm_scale,
                                         cudaStream_t stream) {
  if (!w || count != 34) return KVQ_EINVAL;
  return fp8_paged_attention(
      ptr<void>(w[0]), w[1], w[2], ptr<void>(w[3]), w[4], w[5], i32(w[6]), w[7], w[8], w[9],
      w[10], w[11], ptr<uint8_t>(w[12]), ptr<uint8_t>(w[13]), w[14], w[15], w[16], w[17], w[18],
      ptr<uint8_t>(w[19]), ptr<uint8_t>(w[20]), w[21], ptr<int64_t>(w[22]), w[23], w[24],
      ptr<int64_t>(w[25]), ptr<int64_t>(w[26]), w[27], sm_scale, i32(w[28]), w[29],
      ptr<float>(w[30]), ptr<int32_t>(w[31]), ptr<void>(w[32]), w[33], stream);
}
