// The parts of a row's keys joined: o = sum_s 2^(m_s - m) o_s / sum_s 2^(m_s - m) l_s, m the largest m_s, in the
// parts' order whatever order they ended in.  And the choice of how many parts there are.
#include "paged_attn.h"

namespace svdq {

namespace {

// A wave has a row; lanes over its values, two at a time.
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a) {
  const int64_t rows = (int64_t)a.tokens * a.heads, row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int t = (int)(row / a.heads), h = (int)(row - (int64_t)t * a.heads), lane = threadIdx.x & 63;
  if (t < start_of(a.b, 0, a.tokens) || t >= start_of(a.b, a.b.n, a.tokens)) return;   // no sequence's: left as it is
  const float* ml = a.part + a.splits * rows * a.c.dim + row * a.splits * 2;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; s++) m = fmaxf(m, ml[2 * s]);
  const int dim = a.c.dim;
  float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.splits; s++) {
    const float f = ml[2 * s] == m ? 1.f : __builtin_amdgcn_exp2f(ml[2 * s] - m);
    sum += f * ml[2 * s + 1];
    const float* p = a.part + (s * rows + row) * dim;
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const int d = x * 128 + 2 * lane;
      if (d < dim) {
        o[2 * x] += f * p[d];
        o[2 * x + 1] += f * p[d + 1];
      }
    }
  }
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* to = static_cast<uint16_t*>(a.o) + (int64_t)t * a.o_token + (int64_t)h * a.o_head;
#pragma unroll
  for (int x = 0; x < 2; x++) {
    const int d = x * 128 + 2 * lane;
    if (d < dim) {
      const uint32_t v = pack16(o[2 * x] * f, o[2 * x + 1] * f, a.qbf);
      __builtin_memcpy(to + d, &v, 4);
    }
  }
}

}  // namespace

int attn_splits(int sequences, int tokens, int heads, int kv_heads, int64_t reach) {
  if (sequences <= 0 || tokens <= 0) return 1;
  const int group = heads / kv_heads;
  const int64_t each = ((int64_t)tokens * group + sequences - 1) / sequences;    // rows of a sequence and cache head
  const int64_t tiles = (each + 15) / 16 * sequences * kv_heads;
  int64_t s = 1024 / tiles;
  const int64_t most = reach / 256;
  s = s < most ? s : most;
  return s < 1 ? 1 : s > 128 ? 128 : (int)s;
}

size_t attn_part_bytes(int splits, int tokens, int heads, int dim) {
  return splits <= 1 ? 0 : (size_t)splits * tokens * heads * (dim + 2) * sizeof(float);
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const hipError_t e = attn::launch_few(a, s);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t blocks = ((int64_t)a.tokens * a.heads + 3) / 4;
  if (!launchable(blocks, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(k_attn_join, dim3((unsigned)blocks), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace svdq
