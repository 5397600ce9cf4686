// Causal attention over the 8-bit paged key/value cache (kv8_attention).
#include <math.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "kv8.cuh"

namespace wina {

using namespace kv8;

struct AttnParams {
  kv8_cache_t c;
  const void* q;
  int64_t ld_q;
  int T, Hq, G, shift;
  const int32_t* table;
  int width;
  const int32_t* kv_len;
  const int32_t* cu_q;
  int B, max_q;
  float scale, softcap;
  int window;
  void* out;
  int32_t* status;
};

// One warp per (query, head), keys in order, float32 throughout.
template <bool BF16, bool E4M3, int DH>
__global__ void __launch_bounds__(128) k_kv8_attn_rows(AttnParams p) {
  constexpr int C = DH / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(w / p.Hq), h = (int)(w % p.Hq), g = h / p.G;
  if (p.cu_q && blockIdx.x == 0) {
    for (int x = threadIdx.x; x < p.B; x += 128) {
      const int q0 = __ldg(p.cu_q + x), q1 = __ldg(p.cu_q + x + 1);
      if (q0 < 0 || q1 < q0 || q1 > p.T) record_status(p.status, WINA_ERR_INVALID_ARG);
    }
  }
  if (t >= p.T) return;
  int b = t, i = 0, n = 1;
  if (p.cu_q) {
    int lo = 0, hi = p.B;  // the last request with cu_q <= t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.cu_q + mid) <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int q0 = __ldg(p.cu_q + b), q1 = min(__ldg(p.cu_q + b + 1), p.T);
    if (t < q0 || t >= q1) return;
    i = t - q0;
    n = q1 - q0;
    if (i >= p.max_q) {
      record_status(p.status, WINA_ERR_INVALID_ARG);
      return;
    }
  }
  int kv = __ldg(p.kv_len + b);
  const int room = p.width << p.shift;
  if (kv < 0 || kv > room) {
    record_status(p.status, WINA_ERR_INVALID_ARG);
    kv = max(0, min(kv, room));
  }
  const int pos = kv - n + i;
  const int j0 = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  float q[C], o[C], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < C; ++e) {
    q[e] = load_elem(p.q, BF16 ? WINA_BF16 : WINA_F32, (int64_t)t * p.ld_q + (int64_t)h * DH + lane * C + e);
    o[e] = 0.f;
  }
  for (int j = j0; j <= pos; ++j) {
    const int pg = __ldg(p.table + (int64_t)b * p.width + (j >> p.shift));
    if (pg < 0 || pg >= p.c.n_pages) {
      if (lane == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
      continue;
    }
    const int64_t head = (int64_t)pg * p.c.heads + g;
    const int64_t at = ((head << p.shift) + (j & ((1 << p.shift) - 1))) * DH + lane * C;
    float kf[8], vf[8];
#pragma unroll
    for (int e = 0; e < C; e += 2) {
      float a[4];
      unpack4<E4M3>(*reinterpret_cast<const uint16_t*>((const uint8_t*)p.c.k + at + e), a);
      kf[e] = a[0];
      kf[e + 1] = a[1];
      unpack4<E4M3>(*reinterpret_cast<const uint16_t*>((const uint8_t*)p.c.v + at + e), a);
      vf[e] = a[0];
      vf[e + 1] = a[1];
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < C; ++e) s = fmaf(q[e], kf[e], s);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.c.k_scale[head] * p.scale;
    if (p.softcap > 0.f) s = p.softcap * tanhf(s / p.softcap);
    const float mn = fmaxf(m, s), a = expf(m - mn), e1 = expf(s - mn);
    const float vs = p.c.v_scale[head] * e1;
    l = l * a + e1;
#pragma unroll
    for (int e = 0; e < C; ++e) o[e] = o[e] * a + vs * vf[e];
    m = mn;
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < C; ++e) {
    const int64_t at = ((int64_t)t * p.Hq + h) * DH + lane * C + e;
    if constexpr (BF16) reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o[e] * inv);
    else reinterpret_cast<float*>(p.out)[at] = o[e] * inv;
  }
}

size_t kv8_attention_ws_size(int64_t dh, int64_t rows) {
  (void)dh;
  (void)rows;
  return kAlign;
}

template <bool BF16, bool E4M3>
static void (*rows_kernel(int64_t dh))(AttnParams) {
  return dh == 64 ? k_kv8_attn_rows<BF16, E4M3, 64>
                  : dh == 128 ? k_kv8_attn_rows<BF16, E4M3, 128> : k_kv8_attn_rows<BF16, E4M3, 256>;
}

}  // namespace wina

using namespace wina;

extern "C" wina_status_t kv8_attention(const kv8_cache_t* cache, const void* q, wina_dtype_t qdt, int64_t T,
                                       int64_t ld_q, int64_t Hq, const int32_t* table, int64_t width,
                                       const int32_t* kv_len, const int32_t* cu_q, int64_t B, int64_t max_q,
                                       float scale, int64_t window, float softcap, void* out, void* ws,
                                       size_t ws_bytes, int32_t* status_dev, wina_stream_t stream) {
  const wina_status_t ok = kv8_cache_check(cache);
  if (ok != WINA_OK) return ok;
  if (!valid_dtype(qdt)) return WINA_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || T > (1 << 24) || Hq < 1 || Hq % cache->heads || Hq / cache->heads > 64 || B < 1 || B > kMaxB ||
      max_q < 1 || max_q > (1 << 24) || width < 1 || width > INT32_MAX / cache->page || window < 0 ||
      !(softcap >= 0.f) || !std::isfinite(softcap) || !std::isfinite(scale))
    return WINA_ERR_INVALID_ARG;
  if (!cu_q && (T != B || max_q != 1)) return WINA_ERR_INVALID_ARG;
  if (ld_q < Hq * cache->dh || ld_q > INT32_MAX || ld_q * elem_size(qdt) % 16) return WINA_ERR_INVALID_ARG;
  if (!aligned(status_dev, 4)) return WINA_ERR_INVALID_ARG;
  if (!q || !table || !kv_len || !out || !ws || !aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) ||
      !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(cu_q, 4))
    return WINA_ERR_INVALID_ARG;
  if (ws_bytes < kv8_attention_ws_size(cache->dh, max_q * (Hq / cache->heads))) return WINA_ERR_WORKSPACE;
  if (T == 0) return WINA_OK;
  AttnParams p;
  p.c = *cache;
  p.q = q;
  p.ld_q = ld_q;
  p.T = (int)T;
  p.Hq = (int)Hq;
  p.G = (int)(Hq / cache->heads);
  p.shift = cache->page == 16 ? 4 : cache->page == 32 ? 5 : cache->page == 64 ? 6 : 7;
  p.table = table;
  p.width = (int)width;
  p.kv_len = kv_len;
  p.cu_q = cu_q;
  p.B = (int)B;
  p.max_q = (int)max_q;
  p.scale = scale > 0.f ? scale : (float)(1.0 / std::sqrt((double)cache->dh));
  p.softcap = softcap;
  p.window = (int)std::min<int64_t>(window, INT32_MAX);
  p.out = out;
  p.status = status_dev;
  const bool e4 = cache->format == KV8_E4M3;
  void (*kern)(AttnParams) = qdt == WINA_BF16 ? (e4 ? rows_kernel<true, true>(cache->dh) : rows_kernel<true, false>(cache->dh))
                                              : (e4 ? rows_kernel<false, true>(cache->dh) : rows_kernel<false, false>(cache->dh));
  kern<<<(unsigned)((T * Hq + 3) / 4), 128, 0, (cudaStream_t)stream>>>(p);
  return cuda_status(cudaGetLastError());
}
