// Logits before a token is chosen: penalties for repeated tokens, biases and a
// grammar mask, for a batch of requests with ragged histories.
//
// For token v of request b, with z the logit, c the times v is in the request's
// output and "seen" true if it is in its prompt or output:
//   y = seen ? (z > 0 ? z / rep_b : z * rep_b) : z
//   y = y - freq_b * c - pres_b * [c > 0] + (sum of the biases of v)
//   y = -inf where bit v % 32 of mask word v / 32 is clear
//
// A block takes a slice of one request's vocabulary. It counts the history's
// tokens that fall into the slice in shared memory (bit 31: seen in the prompt;
// the low bits: times in the output; integer atomics, so the counts do not depend
// on their order), then passes over the slice once. Biases come last, each by one
// thread that computes its token anew.
#include <cmath>

#include "vocab.cuh"

namespace embbwd {
namespace {

constexpr int kSlice = 8192;  // tokens of one block
constexpr uint32_t kPromptBit = 0x80000000u;

struct LogitsArgs {
  const void* z;
  void* y;
  int64_t z_stride, y_stride;
  int32_t B, V;
  const int64_t *p_ids, *p_off, *o_ids, *o_off, *b_ids, *b_off;
  int64_t p_n, o_n, b_n;
  const float *rep, *freq, *pres, *b_val;
  const uint32_t* mask;
  int64_t mask_stride;
  uint32_t* status;
};

// [start, end) of request b's list, empty (and reported) if the offsets are malformed.
__device__ __forceinline__ void list_of(const int64_t* off, int64_t n, int32_t b, uint32_t* status, int64_t* start,
                                        int64_t* end) {
  *start = off[b];
  *end = off[b + 1];
  if (*start < 0 || *end < *start || *end > n) {
    report(status, kErrOffsets);
    *start = *end = 0;
  }
}

__device__ __forceinline__ float penalised(float z, uint32_t c, float rep, float freq, float pres) {
  if (c == 0) return z;
  float y = z > 0.f ? __fdiv_rn(z, rep) : z * rep;
  const uint32_t n = c & ~kPromptBit;
  if (n) y = (y - __fmul_rn(freq, (float)n)) - pres;
  return y;
}

template <typename in_t, typename out_t>
__global__ void __launch_bounds__(kThreads) k_logits(LogitsArgs a) {
  __shared__ uint32_t count[kSlice];
  const int32_t b = blockIdx.y;
  const int32_t v0 = blockIdx.x * kSlice, v1 = min(a.V, v0 + kSlice);
  for (int i = threadIdx.x; i < kSlice; i += kThreads) count[i] = 0;
  __syncthreads();
  for (int part = 0; part < 2; ++part) {
    const int64_t* ids = part ? a.o_ids : a.p_ids;
    if (!ids) continue;
    int64_t s, e;
    list_of(part ? a.o_off : a.p_off, part ? a.o_n : a.p_n, b, a.status, &s, &e);
    for (int64_t i = s + threadIdx.x; i < e; i += kThreads) {
      const int64_t v = ids[i];
      if (v < 0 || v >= a.V) {
        report(a.status, kErrIndex);
      } else if (v >= v0 && v < v1) {
        if (part) atomicAdd(&count[v - v0], 1u);
        else atomicOr(&count[v - v0], kPromptBit);
      }
    }
  }
  __syncthreads();
  const float rep = a.rep ? a.rep[b] : 1.f, freq = a.freq ? a.freq[b] : 0.f, pres = a.pres ? a.pres[b] : 0.f;
  const in_t* z = static_cast<const in_t*>(a.z) + b * a.z_stride;
  out_t* y = static_cast<out_t*>(a.y) + b * a.y_stride;
  const uint32_t* mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  int64_t bs = 0, be = 0;
  if (a.b_ids) list_of(a.b_off, a.b_n, b, a.status, &bs, &be);
  for (int32_t v = v0 + threadIdx.x; v < v1; v += kThreads) {
    float x = penalised(Elem<in_t>::get(z[v]), count[v - v0], rep, freq, pres);
    // a token's biases in the order of the list
    for (int64_t j = bs; j < be; ++j)
      if (a.b_ids[j] == v) x += a.b_val[j];
    if (mask && !(mask[v >> 5] >> (v & 31) & 1u)) x = -INFINITY;
    y[v] = Elem<out_t>::put(x);
  }
  for (int64_t j = bs + threadIdx.x; j < be; j += kThreads)
    if (a.b_ids[j] < 0 || a.b_ids[j] >= a.V) report(a.status, kErrIndex);
}

template <typename in_t>
const void* logits_out(int out) {
  switch (out) {
    case EMB_F32: return reinterpret_cast<const void*>(&k_logits<in_t, float>);
    case EMB_F16: return reinterpret_cast<const void*>(&k_logits<in_t, __half>);
    default: return reinterpret_cast<const void*>(&k_logits<in_t, __nv_bfloat16>);
  }
}

const void* logits_kernel(int in, int out) {
  switch (in) {
    case EMB_F32: return logits_out<float>(out);
    case EMB_F16: return logits_out<__half>(out);
    default: return logits_out<__nv_bfloat16>(out);
  }
}

bool list_args_ok(const int64_t* ids, const int64_t* off, int64_t n) {
  if (n < 0 || !aligned(ids, 8) || !aligned(off, 8)) return false;
  return off || (!ids && n == 0);
}

}  // namespace
}  // namespace embbwd

using namespace embbwd;

extern "C" emb_status emb_logits_process(
    int device, const void* logits, emb_dtype logits_dtype, int64_t logits_stride, int32_t B, int32_t V,
    const int64_t* prompt_ids, const int64_t* prompt_offsets, int64_t prompt_n, const int64_t* output_ids,
    const int64_t* output_offsets, int64_t output_n, const float* repetition, const float* frequency,
    const float* presence, const int64_t* bias_ids, const int64_t* bias_offsets, const float* bias_values,
    int64_t bias_n, const uint32_t* mask, int64_t mask_stride, void* out, emb_dtype out_dtype, int64_t out_stride,
    uint32_t* device_status, void* stream) {
  if (device < 0 || B < 0 || B > 65535 || V < 1 || V > kMaxVocab) return EMB_ERR_INVALID_ARG;
  if (!dtype_ok(logits_dtype) || !dtype_ok(out_dtype)) return EMB_ERR_INVALID_ARG;
  if (!list_args_ok(prompt_ids, prompt_offsets, prompt_n) || !list_args_ok(output_ids, output_offsets, output_n) ||
      !list_args_ok(bias_ids, bias_offsets, bias_n) || (bias_ids && !bias_values))
    return EMB_ERR_INVALID_ARG;
  if (!aligned(repetition, 4) || !aligned(frequency, 4) || !aligned(presence, 4) || !aligned(bias_values, 4) ||
      !aligned(mask, 4) || !aligned(device_status, 4))
    return EMB_ERR_INVALID_ARG;
  if (B == 0) return EMB_OK;
  if (!logits || !out || !aligned(logits, dtype_size(logits_dtype)) || !aligned(out, dtype_size(out_dtype)))
    return EMB_ERR_INVALID_ARG;
  if (B > 1 && (logits_stride < V || out_stride < V)) return EMB_ERR_INVALID_ARG;
  if (mask && B > 1 && mask_stride < (V + 31) / 32) return EMB_ERR_INVALID_ARG;
  // in place means the same elements; another type there would be overwritten before it is read
  if (logits == out && (logits_dtype != out_dtype || (B > 1 && logits_stride != out_stride))) return EMB_ERR_INVALID_ARG;
  LogitsArgs a{logits,     out,        logits_stride, out_stride,    B,        V,        prompt_ids, prompt_offsets,
               output_ids, output_offsets, bias_ids,  bias_offsets,  prompt_n, output_n, bias_n,     repetition,
               frequency,  presence,   bias_values,   mask,          mask_stride, device_status};
  return on_device(device, [&] {
    void* args[] = {&a};
    return launch_kernel(logits_kernel(logits_dtype, out_dtype), dim3((V + kSlice - 1) / kSlice, B), dim3(kThreads), 0,
                         static_cast<cudaStream_t>(stream), args, false);
  });
}
