// apa_window.h -- the sliding-window launcher (apa_window.cu) for the C ABI.
#pragma once
#include "apa_internal.h"

namespace apa {
// Exact causal attention with a sliding window and sinks (apa_attention_window): out bf16
// [B,Hq,Nq,d], lse fp32 [B,Hq,Nq] or null; 1 <= window <= Nkv, 0 <= sinks <= Nkv.
cudaError_t launch_window(const Shape& s, const void* q, const void* k, const void* v, int window, int sinks,
                          void* out, float* lse, cudaStream_t st);
}  // namespace apa
