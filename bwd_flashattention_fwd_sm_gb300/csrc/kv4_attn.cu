// Attention over the 4-bit key/value cache.
//
// One warp per query row: its lanes hold the row's values and take the keys one
// after the other, with the running maximum and sum of an online softmax, all in
// float32.
#include "kv4.h"

namespace gbattn {

namespace {

constexpr int kThreads = 128;

template <class T, int D>
__global__ void __launch_bounds__(kThreads) k_kv4_attn(const __grid_constant__ Kv4Args a) {
  constexpr int G = D / kKv4Group, E = D / 32;  // values of a lane
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= (long long)a.batch * a.heads_q * a.seqlen) return;
  const int i = (int)(w % a.seqlen), hq = (int)(w / a.seqlen % a.heads_q), b = (int)(w / a.seqlen / a.heads_q);
  const Kv4Seq s = kv4_seq(a, b);
  if (i >= s.n) return;
  const int pos = s.len - s.n + i, last = a.causal ? pos + 1 : (pos < 0 ? 0 : s.len);
  const T* q = static_cast<const T*>(a.x) + (a.cu ? (s.row0 + i) * a.x_ss : b * a.x_sb + i * a.x_ss) + hq * a.x_sh;
  float qv[E], o[E];
  const int d0 = lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) qv[e] = to_f32(q[d0 + e]), o[e] = 0.f;
  const int g = d0 / kKv4Group, word = (d0 % kKv4Group) / 8 * G + g, shift = d0 % 8 * 4;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < last; ++j) {
    const long long row = kv4_row(a, b, hq / a.group, j);
    if (row < 0) continue;
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(a.kc + row * (D / 2) + word * 4) >> shift;
    const uint32_t vw = *reinterpret_cast<const uint32_t*>(a.vc + row * (D / 2) + word * 4) >> shift;
    const uint32_t ks = a.ks[row * G + g], vs = a.vs[row * G + g];
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      t = fmaf(qv[e], fmaf(bf16_lo(ks), (float)(int)((kw >> (4 * e)) & 15u) - 8.f, bf16_hi(ks)), t);
#pragma unroll
    for (int x = 16; x; x >>= 1) t += __shfl_xor_sync(0xffffffffu, t, x);
    t *= a.scale_log2;
    const float mn = fmaxf(m, t), c = exp2f(m - mn), p = exp2f(t - mn);
    m = mn;
    l = l * c + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(p, fmaf(bf16_lo(vs), (float)(int)((vw >> (4 * e)) & 15u) - 8.f, bf16_hi(vs)), o[e] * c);
  }
  T* y = static_cast<T*>(a.y) + (a.cu ? (s.row0 + i) * a.y_ss : b * a.y_sb + i * a.y_ss) + hq * a.y_sh;
#pragma unroll
  for (int e = 0; e < E; ++e) y[d0 + e] = from_f32<T>(l != 0.f ? o[e] / l : 0.f);
  if (lane == 0)
    a.lse[a.cu ? (long long)hq * a.total + s.row0 + i : ((long long)b * a.heads_q + hq) * a.seqlen + i] =
        l != 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

template <class T, int D>
cudaError_t launch(const Kv4Args& a, cudaStream_t st) {
  const long long rows = (long long)a.batch * a.heads_q * a.seqlen, per = kThreads / 32;
  k_kv4_attn<T, D><<<(unsigned)((rows + per - 1) / per), kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t kv4_attn_workspace(const Kv4Args&, int, bool) { return 0; }

cudaError_t launch_kv4_attn(const Kv4Args& a, int head_dim, bool bf16, void*, cudaStream_t st) {
  if (bf16) {
    if (head_dim == 64) return launch<__nv_bfloat16, 64>(a, st);
    if (head_dim == 128) return launch<__nv_bfloat16, 128>(a, st);
    return launch<__nv_bfloat16, 256>(a, st);
  }
  if (head_dim == 64) return launch<float, 64>(a, st);
  if (head_dim == 128) return launch<float, 128>(a, st);
  return launch<float, 256>(a, st);
}

}  // namespace gbattn
