// The 8-bit paged key/value cache: where a step's tokens go (kv8_plan), their rows into the
// pages (kv8_write) and back (kv8_read).
#include <cooperative_groups.h>

#include <algorithm>

#include "internal.h"
#include "kv8.cuh"

namespace wina {

using namespace kv8;

// ------------------------------------------------------------------------------------
// kv8_plan
// ------------------------------------------------------------------------------------

constexpr int kPlanT = 512;         // threads per CTA
constexpr int kPlanCtas = 8;        // CTAs of the cluster that shares a large plan
constexpr int64_t kPlanOne = 4096;  // tokens up to which one CTA does it all

struct PlanParams {
  const int32_t* seq_len;
  const int32_t* new_len;
  int B, shift;  // page = 1 << shift
  int32_t* table;
  int width;
  int32_t* free_pages;
  int cells;
  const int32_t* n_free;
  int tokens;
  int32_t *kv_len, *cu_q, *slots, *positions, *n_free_out, *status;
};

struct Sum3 {
  long long a, b, c;
};

// Exclusive prefix sums of three counts per thread over the block; `total` gets the sums.
// Three barriers.
__device__ __forceinline__ Sum3 block_scan3(Sum3 v, Sum3* red, Sum3* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sum3 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o),
                    c = __shfl_up_sync(0xffffffffu, x.c, o);
    if (lane >= o) {
      x.a += a;
      x.b += b;
      x.c += c;
    }
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0 && lane < kPlanT / 32) {
    Sum3 w = red[lane];
#pragma unroll
    for (int o = 1; o < kPlanT / 32; o <<= 1) {
      const unsigned m = (1u << (kPlanT / 32)) - 1u;
      const long long a = __shfl_up_sync(m, w.a, o), b = __shfl_up_sync(m, w.b, o), c = __shfl_up_sync(m, w.c, o);
      if (lane >= o) {
        w.a += a;
        w.b += b;
        w.c += c;
      }
    }
    red[lane] = w;
  }
  __syncthreads();
  *total = red[kPlanT / 32 - 1];
  if (warp) {
    x.a += red[warp - 1].a;
    x.b += red[warp - 1].b;
    x.c += red[warp - 1].c;
  }
  __syncthreads();
  return Sum3{x.a - v.a, x.b - v.b, x.c - v.c};
}

// The last b in [0, n) with p[b] <= v (p ascending, p[0] <= v).
__device__ __forceinline__ int last_at_most(const int32_t* p, int n, int v) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int sat32(long long v) { return (int)(v > 0x7fffffffLL ? 0x7fffffffLL : v); }

// One cluster (or one CTA for a small plan). Every CTA makes the prefix sums over the
// requests for itself in shared memory (three loads deep, no exchange); the tokens, the new
// table entries and the pushed cells are then shared out over the cluster's threads, each
// finding its request by a binary search. A page that was popped is computed from the stack
// wherever it is needed, never read back from the table, and cells are read below *n_free
// and written from there on, so only the outputs that may overlay inputs (kv_len, n_free_out)
// wait for the cluster's barrier. Latency-bound: the work is two dependent loads, a scan and
// the stores.
__global__ void __launch_bounds__(kPlanT) k_kv8_plan(PlanParams p) {
  extern __shared__ int32_t psm[];
  __shared__ Sum3 red[kPlanT / 32];
  __shared__ int s_taken;
  const int tid = threadIdx.x, B = p.B, page = 1 << p.shift;
  int32_t* tok = psm;              // [B + 1] tokens before request b
  int32_t* need = tok + B + 1;     // [B + 1] pages popped before it
  int32_t* back = need + B + 1;    // [B + 1] pages pushed before it
  int32_t* seq = back + B + 1;     // [B] cached tokens; ~(clamped) for a request left out
  const int room = (int)min((long long)p.width << p.shift, 0x7fffffffLL);
  int n_free = *p.n_free;
  if (tid == 0) s_taken = 0;
  Sum3 run = {0, 0, 0};
  for (int b0 = 0; b0 < B; b0 += kPlanT) {
    const int b = b0 + tid;
    Sum3 v = {0, 0, 0};
    int sq = 0;
    if (b < B) {
      sq = p.seq_len[b];
      const int nw = p.new_len[b];
      const bool bad = sq < 0 || sq > room || (nw > 0 && nw > room - sq);
      const int have = bad ? 0 : (sq + page - 1) >> p.shift;
      v.a = max(nw, 0);
      if (!bad) {
        if (nw < 0) v.c = have;
        else v.b = (int)(((long long)sq + nw + page - 1) >> p.shift) - have;
      }
      if (bad) {
        sq = ~max(0, min(sq, room));
        if (blockIdx.x == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
      }
    }
    Sum3 tot;
    const Sum3 ex = block_scan3(v, red, &tot);
    if (b < B) {
      tok[b] = sat32(run.a + ex.a);
      need[b] = sat32(run.b + ex.b);
      back[b] = sat32(run.c + ex.c);
      seq[b] = sq;
    }
    run.a += tot.a;
    run.b += tot.b;
    run.c += tot.c;
  }
  if (tid == 0) {
    tok[B] = sat32(run.a);
    need[B] = sat32(run.b);
    back[B] = sat32(run.c);
  }
  if (n_free < 0 || n_free > p.cells) {
    if (blockIdx.x == 0 && tid == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
    n_free = max(0, min(n_free, p.cells));
  }
  __syncthreads();
  const long long want_top = (long long)n_free + run.c;
  const int top = (int)min(want_top, (long long)p.cells), pushed = top - n_free;
  if (want_top > p.cells && blockIdx.x == 0 && tid == 0) record_status(p.status, WINA_ERR_CAPACITY);
  // whether request b gets its places; its tokens' prefix sums are exact if it does
  auto served = [&](int b) { return seq[b] >= 0 && need[b + 1] <= top && tok[b + 1] <= p.tokens; };
  // the r-th page pushed
  auto pushed_page = [&](int r) {
    const int b = last_at_most(back, B, r);
    return p.table[(int64_t)b * p.width + (r - back[b])];
  };
  // the j-th page popped
  auto popped_page = [&](int j) {
    const int e = top - 1 - j;
    return e < n_free ? p.free_pages[e] : pushed_page(e - n_free);
  };
  const int ctas = gridDim.x, rank = blockIdx.x;
  // tokens, four to a thread
  for (int64_t t0 = 4 * ((int64_t)rank * kPlanT + tid); t0 < p.tokens; t0 += 4LL * ctas * kPlanT) {
    int sl[4], ps[4];
    int b = B;
    if (t0 < tok[B]) b = last_at_most(tok, B, (int)t0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + i;
      sl[i] = -1;
      ps[i] = 0;
      if (t >= p.tokens) continue;
      while (b < B && t >= tok[b + 1]) ++b;
      if (b < B && served(b)) {
        const int pos = seq[b] + (int)t - tok[b], pi = pos >> p.shift, have = (seq[b] + page - 1) >> p.shift;
        const int pg = pi < have ? p.table[(int64_t)b * p.width + pi] : popped_page(need[b] + pi - have);
        if (pg >= 0 && pg <= (0x7fffffff >> p.shift)) {
          sl[i] = (pg << p.shift) | (pos & (page - 1));
          ps[i] = pos;
        }
      }
    }
    if (t0 + 4 <= p.tokens) {
      *reinterpret_cast<int4*>(p.slots + t0) = make_int4(sl[0], sl[1], sl[2], sl[3]);
      if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(ps[0], ps[1], ps[2], ps[3]);
    } else {
      for (int i = 0; t0 + i < p.tokens; ++i) {
        p.slots[t0 + i] = sl[i];
        if (p.positions) p.positions[t0 + i] = ps[i];
      }
    }
  }
  // the pages popped and served go behind their request's present ones
  for (int j = rank * kPlanT + tid; j < min(need[B], top); j += ctas * kPlanT) {
    const int b = last_at_most(need, B, j);
    if (served(b)) {
      const int have = (seq[b] + page - 1) >> p.shift;
      p.table[(int64_t)b * p.width + have + (j - need[b])] = popped_page(j);
    }
  }
  for (int r = rank * kPlanT + tid; r < pushed; r += ctas * kPlanT) p.free_pages[n_free + r] = pushed_page(r);
  // what may overlay the inputs: after every CTA has read them
  if (ctas > 1) cooperative_groups::this_cluster().sync();
  for (int b = rank * kPlanT + tid; b < B; b += ctas * kPlanT) {
    const bool ended = back[b + 1] > back[b];
    const int n = tok[b + 1] - tok[b];
    int kv = seq[b] < 0 ? ~seq[b] : (ended ? 0 : seq[b]);
    if (!ended && served(b)) kv += n;
    else if (seq[b] >= 0 && n > 0) record_status(p.status, WINA_ERR_CAPACITY);
    p.kv_len[b] = kv;
    p.cu_q[b] = min(tok[b], p.tokens);
  }
  if (rank == 0) {
    for (int b = tid; b < B; b += kPlanT)
      if (served(b)) atomicMax(&s_taken, need[b + 1]);
    __syncthreads();
    if (tid == 0) {
      p.cu_q[B] = min(tok[B], p.tokens);
      *p.n_free_out = top - s_taken;
    }
  }
}

// ------------------------------------------------------------------------------------
// kv8_write
// ------------------------------------------------------------------------------------

constexpr int kWriteW = 8;      // warps per CTA
constexpr int kWriteSeg = 16;   // tokens a CTA looks for runs in, at most

struct WriteParams {
  kv8_cache_t c;
  const void* x[2];   // keys, values
  int64_t ld[2];
  const int32_t* slots;
  int T, seg, shift;
  int32_t* status;
};

// One warp per (run of rows in one page, head, keys or values): the rows' largest magnitude,
// the scale, the bytes. DH / 8 lanes hold a row, eight channels each, so a pass over up to
// kRows rows has all its 16-byte loads in flight; a run longer than that is read twice, the
// second time from L1/L2. Bound by HBM for prompts (each element read once, one byte
// written), by latency for single tokens.
template <bool BF16, bool E4M3, int DH>
__global__ void __launch_bounds__(32 * kWriteW) k_kv8_write(WriteParams p) {
  constexpr int LPR = DH / 8, RPP = 32 / LPR;  // lanes per row, rows per pass
  constexpr int IT = BF16 ? 8 : 4;             // passes held in registers
  __shared__ int s_run[kWriteSeg], s_n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t0 = blockIdx.x * p.seg, page = 1 << p.shift;
  const int64_t limit = p.c.n_pages << p.shift;
  if (warp == 0) {
    const int t = t0 + lane;
    bool start = false;
    if (lane < p.seg && t < p.T) {
      const int s = __ldg(p.slots + t);
      if (s >= limit) record_status(p.status, WINA_ERR_INVALID_ARG);
      start = s >= 0 && s < limit && ((s & (page - 1)) == 0 || t == 0 || __ldg(p.slots + t - 1) != s - 1);
    }
    const unsigned m = __ballot_sync(0xffffffffu, start);
    if (start) s_run[__popc(m & ((1u << lane) - 1u))] = t;
    if (lane == 0) s_n = __popc(m);
  }
  __syncthreads();
  const int H2 = 2 * (int)p.c.heads, items = s_n * H2;
  const int sub = lane / LPR, ch = (lane % LPR) * 8;
  for (int it = blockIdx.y * kWriteW + warp; it < items; it += gridDim.y * kWriteW) {
    const int t = s_run[it / H2], which = (it % H2) / (int)p.c.heads, h = (it % H2) % (int)p.c.heads;
    const int slot = __ldg(p.slots + t), first = slot & (page - 1), pg = slot >> p.shift;
    // the run: consecutive tokens at consecutive places of the page
    int len = 1;
    for (int base = 1; base < page - first; base += 32) {
      const int i = base + lane;
      const bool on = i < page - first && t + i < p.T && __ldg(p.slots + t + i) == slot + i;
      const unsigned m = __ballot_sync(0xffffffffu, on);
      const int more = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      len += more;
      if (more < 32) break;
    }
    const void* x = which ? p.x[1] : p.x[0];
    const int64_t ld = which ? p.ld[1] : p.ld[0], src = (int64_t)t * ld + (int64_t)h * DH + ch;
    float* scale_at = (which ? p.c.v_scale : p.c.k_scale) + (int64_t)pg * p.c.heads + h;
    uint8_t* dst = reinterpret_cast<uint8_t*>(which ? p.c.v : p.c.k) + (((int64_t)pg * p.c.heads + h) << p.shift) * DH + ch;
    const float present = first ? *scale_at : 0.f;
    Row8<BF16> r[IT];
    uint32_t amax = 0;  // magnitudes order like their bits, NaN above all
    for (int i0 = 0; i0 < len; i0 += IT * RPP) {
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        const int i = i0 + q * RPP + sub;
        if (i < len) r[q].load(x, src + (int64_t)i * ld);
      }
#pragma unroll
      for (int q = 0; q < IT; ++q)
        if (i0 + q * RPP + sub < len) {
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(r[q].get(e)) & 0x7fffffffu);
        }
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
    float s;
    bool void_ = amax >= 0x7f800000u || present != present;  // no scale holds these rows
    if (void_) {
      s = __uint_as_float(0x7fc00000u);
    } else {
      s = pow2_scale<E4M3>(amax);
      if (first && present > s) s = present;
    }
    if (first && !void_ && s != present) {
      // the scale grew: the page's older rows, rounded again
      const float f = __fdiv_rn(present, s);
      for (int i = sub; i < first; i += RPP) {
        uint2 w = *reinterpret_cast<const uint2*>(dst + i * DH);
        float a[4], b[4];
        unpack4<E4M3>(w.x, a);
        unpack4<E4M3>(w.y, b);
        w.x = pack4<E4M3>(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
        w.y = pack4<E4M3>(b[0] * f, b[1] * f, b[2] * f, b[3] * f);
        *reinterpret_cast<uint2*>(dst + i * DH) = w;
      }
    }
    const float inv = void_ ? 0.f : __fdiv_rn(1.f, s);
    const bool again = len > IT * RPP;
    for (int i0 = 0; i0 < len; i0 += IT * RPP) {
      if (again) {
#pragma unroll
        for (int q = 0; q < IT; ++q) {
          const int i = i0 + q * RPP + sub;
          if (i < len) r[q].load(x, src + (int64_t)i * ld);
        }
      }
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        const int i = i0 + q * RPP + sub;
        if (i < len) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = void_ ? 0.f : r[q].get(e) * inv;
          const uint2 w = make_uint2(pack4<E4M3>(v[0], v[1], v[2], v[3]), pack4<E4M3>(v[4], v[5], v[6], v[7]));
          *reinterpret_cast<uint2*>(dst + (first + i) * DH) = w;
        }
      }
    }
    if (lane == 0 && (first == 0 || s != present)) *scale_at = s;
  }
}

// ------------------------------------------------------------------------------------
// kv8_read
// ------------------------------------------------------------------------------------

struct ReadParams {
  kv8_cache_t c;
  const int32_t* slots;
  void* out[2];
  int64_t pieces;  // 16-channel pieces of one of the two
  int shift, log_row;  // pieces of a head's row: 1 << log_row
  int32_t* status;
};

// 16 channels per thread: one 16-byte load, two (bf16) or four (float32) 16-byte stores.
// HBM-bound; a page's place is found once per piece, from L1.
template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(256) k_kv8_read(ReadParams p) {
  const int64_t limit = p.c.n_pages << p.shift;
  const int which = blockIdx.y;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(which ? p.c.v : p.c.k);
  const float* scales = which ? p.c.v_scale : p.c.k_scale;
  void* const out = which ? p.out[1] : p.out[0];
  if (!out) return;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.pieces; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i >> p.log_row;  // token * heads + head
    const int64_t t = row / p.c.heads;
    const int h = (int)(row - t * p.c.heads);
    const int s = __ldg(p.slots + t);
    float f[16];
    if (s >= 0 && s < limit) {
      const int pg = s >> p.shift, off = s & ((1 << p.shift) - 1);
      const int64_t head = (int64_t)pg * p.c.heads + h;
      const uint4 w = *reinterpret_cast<const uint4*>(src + ((((head << p.shift) + off) << p.log_row) + (i & ((1 << p.log_row) - 1))) * 16);
      const float sc = scales[head];
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float a[4];
        unpack4<E4M3>(u[q], a);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[4 * q + e] = a[e] * sc;
      }
    } else {
      if (s >= limit) record_status(p.status, WINA_ERR_INVALID_ARG);
#pragma unroll
      for (int e = 0; e < 16; ++e) f[e] = 0.f;
    }
    if constexpr (BF16) {
      uint4* d = reinterpret_cast<uint4*>(out) + i * 2;
      uint32_t o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        o[e] = *reinterpret_cast<const uint32_t*>(&b);
      }
      d[0] = make_uint4(o[0], o[1], o[2], o[3]);
      d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else {
      float4* d = reinterpret_cast<float4*>(out) + i * 4;
#pragma unroll
      for (int q = 0; q < 4; ++q) d[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
    }
  }
}

static int page_shift(int64_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

static bool page_ok(int64_t page) { return page == 16 || page == 32 || page == 64 || page == 128; }

wina_status_t kv8_cache_check(const kv8_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return WINA_ERR_INVALID_ARG;
  if (c->format != KV8_INT8 && c->format != KV8_E4M3) return WINA_ERR_UNSUPPORTED_DTYPE;
  if (!page_ok(c->page) || (c->dh != 64 && c->dh != 128 && c->dh != 256)) return WINA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_pages > INT32_MAX / c->page || c->heads < 1 || c->heads > 1024) return WINA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4))
    return WINA_ERR_INVALID_ARG;
  return WINA_OK;
}

}  // namespace wina

using namespace wina;

extern "C" wina_status_t kv8_plan(const int32_t* seq_len, const int32_t* new_len, int64_t B, int64_t page,
                                  int32_t* table, int64_t width, int32_t* free_pages, int64_t cells,
                                  const int32_t* n_free, int64_t tokens, int32_t* kv_len, int32_t* cu_q,
                                  int32_t* slots, int32_t* positions, int32_t* n_free_out, int32_t* status_dev,
                                  wina_stream_t stream) {
  if (B < 1 || B > kMaxB || !page_ok(page) || width < 1 || width > INT32_MAX / page || cells < 1 ||
      cells > (1 << 30) || tokens < 0 || tokens > (1 << 30))
    return WINA_ERR_INVALID_ARG;
  if (!seq_len || !new_len || !table || !free_pages || !n_free || !kv_len || !cu_q || (tokens && !slots) || !n_free_out)
    return WINA_ERR_INVALID_ARG;
  const void* four[] = {seq_len, new_len, table, free_pages, n_free, kv_len, cu_q, n_free_out, status_dev};
  for (const void* q : four)
    if (!aligned(q, 4)) return WINA_ERR_INVALID_ARG;
  if (!aligned(slots, 16) || !aligned(positions, 16)) return WINA_ERR_INVALID_ARG;
  PlanParams p = {seq_len,     new_len,    (int)B,   page_shift(page), table, (int)width, free_pages, (int)cells, n_free,
                  (int)tokens, kv_len, cu_q,     slots,            positions, n_free_out, status_dev};
  const size_t smem = (size_t)(4 * B + 3) * 4;
  cudaError_t e = ensure_smem_limit((const void*)k_kv8_plan, smem);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  const int ctas = tokens <= kPlanOne ? 1 : kPlanCtas;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k_kv8_plan, p));
}

template <bool BF16, bool E4M3>
static void (*write_kernel(int64_t dh))(WriteParams) {
  return dh == 64 ? k_kv8_write<BF16, E4M3, 64> : dh == 128 ? k_kv8_write<BF16, E4M3, 128> : k_kv8_write<BF16, E4M3, 256>;
}

extern "C" wina_status_t kv8_write(const kv8_cache_t* cache, const void* k, const void* v, wina_dtype_t xdt, int64_t T,
                                   int64_t ld_k, int64_t ld_v, const int32_t* slots, int32_t* status_dev,
                                   wina_stream_t stream) {
  const wina_status_t ok = kv8_cache_check(cache);
  if (ok != WINA_OK) return ok;
  if (!valid_dtype(xdt)) return WINA_ERR_UNSUPPORTED_DTYPE;
  const int64_t row = cache->heads * cache->dh, es = elem_size(xdt);
  if (T < 0 || T > (1 << 30) || ld_k < row || ld_v < row || ld_k > INT32_MAX || ld_v > INT32_MAX || ld_k * es % 16 ||
      ld_v * es % 16)
    return WINA_ERR_INVALID_ARG;
  if (!aligned(status_dev, 4)) return WINA_ERR_INVALID_ARG;
  if (T == 0) return WINA_OK;
  if (!k || !v || !slots || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4)) return WINA_ERR_INVALID_ARG;
  WriteParams p;
  p.c = *cache;
  p.x[0] = k;
  p.x[1] = v;
  p.ld[0] = ld_k;
  p.ld[1] = ld_v;
  p.slots = slots;
  p.T = (int)T;
  p.shift = page_shift(cache->page);
  p.status = status_dev;
  // few tokens: one to a CTA, and the heads over several, so that single tokens' pages are
  // written side by side; many: kWriteSeg to a CTA
  const int64_t sms = device_sm_count();
  if (sms < 1) return WINA_ERR_CUDA;
  p.seg = (int)std::max<int64_t>(1, std::min<int64_t>(kWriteSeg, T / sms));
  const int64_t gx = (T + p.seg - 1) / p.seg, most = 2 * cache->heads;
  const int64_t gy = (most + kWriteW - 1) / kWriteW;
  const bool e4 = cache->format == KV8_E4M3;
  void (*kern)(WriteParams) = xdt == WINA_BF16 ? (e4 ? write_kernel<true, true>(cache->dh) : write_kernel<true, false>(cache->dh))
                                               : (e4 ? write_kernel<false, true>(cache->dh) : write_kernel<false, false>(cache->dh));
  kern<<<dim3((unsigned)gx, (unsigned)gy), 32 * kWriteW, 0, (cudaStream_t)stream>>>(p);
  return cuda_status(cudaGetLastError());
}

extern "C" wina_status_t kv8_read(const kv8_cache_t* cache, const int32_t* slots, int64_t T, void* k, void* v,
                                  wina_dtype_t xdt, int32_t* status_dev, wina_stream_t stream) {
  const wina_status_t ok = kv8_cache_check(cache);
  if (ok != WINA_OK) return ok;
  if (!valid_dtype(xdt)) return WINA_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || T > (1 << 30) || !aligned(status_dev, 4) || !aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16))
    return WINA_ERR_INVALID_ARG;
  if (T == 0 || (!k && !v)) return WINA_OK;
  if (!slots) return WINA_ERR_INVALID_ARG;
  ReadParams p;
  p.c = *cache;
  p.slots = slots;
  p.out[0] = k;
  p.out[1] = v;
  p.log_row = cache->dh == 64 ? 2 : cache->dh == 128 ? 3 : 4;
  p.pieces = T * cache->heads << p.log_row;
  p.shift = page_shift(cache->page);
  p.status = status_dev;
  const int sms = device_sm_count();
  if (sms < 1) return WINA_ERR_CUDA;
  const dim3 grid((unsigned)std::min<int64_t>((p.pieces + 255) / 256, (int64_t)sms * 16), 2);
  const bool e4 = cache->format == KV8_E4M3;
  void (*kern)(ReadParams) = xdt == WINA_BF16 ? (e4 ? k_kv8_read<true, true> : k_kv8_read<true, false>)
                                              : (e4 ? k_kv8_read<false, true> : k_kv8_read<false, false>);
  kern<<<grid, 256, 0, (cudaStream_t)stream>>>(p);
  return cuda_status(cudaGetLastError());
}
