// How the streaming norm kernels (norm.cu) fill an SM: threads, CTAs, and stages of rows in shared memory.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kNormStages = 8;           // rows on their way at most
constexpr int kNormSmem = 212 << 10;     // per SM, for the stages
constexpr int kSmSmem = 228 << 10;       // all of an SM's shared memory
constexpr int kCtaSmem = 1024 + 512;     // of which each CTA has the runtime's reserve, and barriers and sums, beside its stages
constexpr int kRowVpt = 2;               // 8-column chunks of a row per thread, forward
constexpr int kRowThreadsPerSm = 1024;   // 64 registers each
constexpr int kGradVpt = 2;              // and backward
constexpr int kGradNw = 16;              // warps per SM: 128 registers a thread

constexpr int row_threads(int nv) { return (nv + 31) / 32 * 32; }

// CTAs per SM for rows of nv chunks.
constexpr int row_ctas(int nv) {
  const int n = kRowThreadsPerSm / row_threads((nv + kRowVpt - 1) / kRowVpt);
  return n < 1 ? 1 : (n < 16 ? n : 16);
}
constexpr int grad_ctas(int nv) {
  const int n = kGradNw * 32 / row_threads((nv + kGradVpt - 1) / kGradVpt);
  return n < 8 ? n : 8;
}

// Bytes of stages of one of `ctas` CTAs: their share, and no more than lets all of them be resident.  (With 1 / 16 of
// kNormSmem each, rows of 832 to 848 and 944 to 968 bf16 columns had 15 of 16 CTAs resident, and the
// last 152 of 2432 ran a round of their own: 16384 x 960 20.0 us, 16384 x 976 16.7.)
constexpr int stage_room(int ctas) {
  const int share = kNormSmem / ctas, most = kSmSmem / ctas - kCtaSmem;
  return share < most ? share : most;
}

// Stages of a CTA with `bytes` in each.
constexpr int norm_stages(int ctas, int64_t bytes) {
  const int64_t n = stage_room(ctas) / bytes;
  return n < kNormStages ? (int)n : kNormStages;
}

}  // namespace moe
