// experts_words.cu — the operators around a layer of experts, called with their
// arguments as an array of 64-bit words (a binding that converts arguments one
// by one pays for each).
#include <cstdint>

#include "kvq_experts.h"

namespace {

template <typename T>
T* ptr(int64_t w) {
  return reinterpret_cast<T*>(static_cast<uintptr_t>(w));
}

// A 32-bit argument; one that does not fit becomes a value that the functions
// refuse.
int32_t i32(int64_t w) { return w < -1 || w > INT32_MAX ? -1 : static_cast<int32_t>(w); }

}  // namespace

extern "C" int fp8_matmul_words(const int64_t* w, int64_t count, cudaStream_t stream) {
  if (!w || count != 22) return KVQ_EINVAL;
  return fp8_matmul(ptr<uint8_t>(w[0]), w[1], ptr<float>(w[2]), w[3], w[4], w[5],
                    ptr<uint8_t>(w[6]), w[7], w[8], ptr<float>(w[9]), w[10], w[11], w[12], w[13],
                    w[14], ptr<int64_t>(w[15]), ptr<int64_t>(w[16]), w[17], ptr<void>(w[18]),
                    w[19], i32(w[20]), ptr<int32_t>(w[21]), stream);
}

extern "C" int fp8_gated_matmul_words(const int64_t* w, int64_t count, cudaStream_t stream) {
  if (!w || count != 23) return KVQ_EINVAL;
  return fp8_gated_matmul(ptr<uint8_t>(w[0]), w[1], ptr<float>(w[2]), w[3], w[4], w[5],
                          ptr<uint8_t>(w[6]), w[7], w[8], ptr<float>(w[9]), w[10], w[11], w[12],
                          w[13], w[14], ptr<int64_t>(w[15]), ptr<int64_t>(w[16]), w[17],
                          ptr<uint8_t>(w[18]), w[19], ptr<float>(w[20]), w[21],
                          ptr<int32_t>(w[22]), stream);
}

extern "C" int route_experts_words(const int64_t* w, int64_t count, float scale,
                                   cudaStream_t stream) {
  if (!w || count != 13) return KVQ_EINVAL;
  return route_experts(ptr<void>(w[0]), w[1], i32(w[2]), w[3], w[4], w[5], i32(w[6]),
                       ptr<float>(w[7]), w[8], w[9], i32(w[10]), scale, ptr<int64_t>(w[11]),
                       ptr<float>(w[12]), stream);
}

extern "C" int sort_by_expert_words(const int64_t* w, int64_t count, cudaStream_t stream) {
  if (!w || count != 9) return KVQ_EINVAL;
  return sort_by_expert(ptr<int64_t>(w[0]), w[1], w[2], w[3], ptr<int64_t>(w[4]),
                        ptr<int64_t>(w[5]), ptr<int64_t>(w[6]), ptr<void>(w[7]), w[8], stream);
}

extern "C" int combine_experts_words(const int64_t* w, int64_t count, cudaStream_t stream) {
  if (!w || count != 13) return KVQ_EINVAL;
  return combine_experts(ptr<void>(w[0]), w[1], w[2], ptr<int64_t>(w[3]), ptr<float>(w[4]), w[5],
                         w[6], ptr<void>(w[7]), w[8], ptr<void>(w[9]), w[10], w[11], i32(w[12]),
                         stream);
}
