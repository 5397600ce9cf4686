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
  // a thread's consecutive requests, then one scan over the threads
  const int per = (B + kPlanT - 1) / kPlanT, b_lo = min(tid * per, B), b_hi = min(b_lo + per, B);
  Sum3 mine = {0, 0, 0};
#pragma unroll 4
  for (int b = b_lo; b < b_hi; ++b) {
    int sq = p.seq_len[b];
    const int nw = p.new_len[b];
    const bool bad = sq < 0 || sq > room || (nw > 0 && nw > room - sq);
    const int have = bad ? 0 : (sq + page - 1) >> p.shift;
    mine.a += max(nw, 0);
    if (!bad) {
      if (nw < 0) mine.c += have;
      else mine.b += (int)(((long long)sq + nw + page - 1) >> p.shift) - have;
    } else {
      sq = ~max(0, min(sq, room));
      if (blockIdx.x == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
    }
    // inclusive within the thread for now
    tok[b + 1] = sat32(mine.a);
    need[b + 1] = sat32(mine.b);
    back[b + 1] = sat32(mine.c);
    seq[b] = sq;
  }
  Sum3 run;
  const Sum3 ex = block_scan3(mine, red, &run);
  for (int b = b_lo; b < b_hi; ++b) {
    tok[b + 1] = sat32(ex.a + tok[b + 1]);
    need[b + 1] = sat32(ex.b + need[b + 1]);
    back[b + 1] = sat32(ex.c + back[b + 1]);
  }
  if (tid == 0) tok[0] = need[0] = back[0] = 0;
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
  // where the r-th page pushed, and the j-th page popped, are read
  auto pushed_at = [&](int r) -> const int32_t* {
    const int b = last_at_most(back, B, r);
    return p.table + (int64_t)b * p.width + (r - back[b]);
  };
  auto popped_at = [&](int j) {
    const int e = top - 1 - j;
    return e < n_free ? p.free_pages + e : pushed_at(e - n_free);
  };
  const int ctas = gridDim.x, rank = blockIdx.x;
  // tokens, four to a thread
  for (int64_t t0 = 4 * ((int64_t)rank * kPlanT + tid); t0 < p.tokens; t0 += 4LL * ctas * kPlanT) {
    int sl[4], ps[4], pg[4];
    const int32_t* at[4];
    int b = B;
    if (t0 < tok[B]) b = last_at_most(tok, B, (int)t0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // first where the pages are read, then all four at once
      const int64_t t = t0 + i;
      at[i] = nullptr;
      ps[i] = 0;
      if (t >= p.tokens) continue;
      while (b < B && t >= tok[b + 1]) ++b;
      if (b < B && served(b)) {
        const int pos = seq[b] + (int)t - tok[b], pi = pos >> p.shift, have = (seq[b] + page - 1) >> p.shift;
        at[i] = pi < have ? p.table + (int64_t)b * p.width + pi : popped_at(need[b] + pi - have);
        ps[i] = pos;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) pg[i] = at[i] ? *at[i] : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool ok = pg[i] >= 0 && pg[i] <= (0x7fffffff >> p.shift);
      sl[i] = ok ? (pg[i] << p.shift) | (ps[i] & (page - 1)) : -1;
      if (!ok) ps[i] = 0;
      if (!ok && at[i]) record_status(p.status, WINA_ERR_INVALID_ARG);  // a table or stack entry that is no page
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
      p.table[(int64_t)b * p.width + have + (j - need[b])] = *popped_at(j);
    }
  }
  // (the last threads first: the first ones have the tokens)
  for (int r0 = (ctas - 1 - rank) * kPlanT + (kPlanT - 1 - tid); r0 < pushed; r0 += 4 * ctas * kPlanT) {
    // four at a time: their searches and loads do not wait for one another
    int pg[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * ctas * kPlanT;
      pg[u] = r < pushed ? *pushed_at(r) : 0;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = r0 + u * ctas * kPlanT;
      if (r < pushed) p.free_pages[n_free + r] = pg[u];
    }
  }
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
// IT * RPP rows has all its 16-byte loads in flight; a run longer than that is read twice, the
// second time from L1/L2. Bound by HBM for prompts (each element read once, one byte
// written), by latency for single tokens. Four CTAs of 64 registers share an SM: with more rows
// in registers, or the runs' lengths found beforehand, 15500 bf16 rows of 8 x 128 in pages of 32
// took 29 to 44 us instead of 25.
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
    bool lost = amax >= 0x7f800000u || present != present;  // no scale holds these rows
    if (lost) {
      s = __uint_as_float(0x7fc00000u);
    } else {
      s = pow2_scale<E4M3>(amax);
      if (first && present > s) s = present;
    }
    if (first && !lost && s != present) {
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
    const float inv = lost ? 0.f : __fdiv_rn(1.f, s);
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
          for (int e = 0; e < 8; ++e) v[e] = lost ? 0.f : r[q].get(e) * inv;
          const uint2 w = make_uint2(pack4<E4M3>(v[0], v[1], v[2], v[3]), pack4<E4M3>(v[4], v[5], v[6], v[7]));
          *reinterpret_cast<uint2*>(dst + (first + i) * DH) = w;
        }
      }
    }
    if (lane == 0 && (first == 0 || s != present)) *scale_at = s;
    if (const uint32_t limit = byte_limit<E4M3>(s)) {
      __syncwarp();
      limit_rows<E4M3, DH>(dst, (s == present ? first : 0) + sub, RPP, first + len, limit);
    }
  }
}

// The same where a page is more than four times what a warp holds: its longer runs
// are shared by the CTA's eight warps, which exchange their maxima; the shorter ones are one
// warp's. (3010 float32 rows of 4 x 256 in pages of 64: 28 us with a warp to an item, 12 us so;
// with eight warps to each run of 32 bf16 rows of 128, which two hold, 80 us instead of 25.)
template <bool BF16, bool E4M3, int DH>
__global__ void __launch_bounds__(32 * kWriteW, 3) k_kv8_write_shared(WriteParams p) {
  constexpr int LPR = DH / 8, RPP = 32 / LPR;  // lanes per row, rows per pass
  constexpr int IT = BF16 ? 8 : 4;             // passes held in registers
  constexpr int ROWS = IT * RPP;               // rows a warp holds
  __shared__ int s_run[kWriteSeg], s_len[kWriteSeg], s_n;
  __shared__ uint32_t s_amax[kWriteW];
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
  // the runs' lengths: consecutive tokens at consecutive places of the page
  for (int r = warp; r < s_n; r += kWriteW) {
    const int t = s_run[r], slot = __ldg(p.slots + t), first = slot & (page - 1);
    int len = 1;
    for (int base = 1; base < page - first; base += 32) {
      const int i = base + lane;
      const bool on = i < page - first && t + i < p.T && __ldg(p.slots + t + i) == slot + i;
      const unsigned m = __ballot_sync(0xffffffffu, on);
      const int more = m == 0xffffffffu ? 32 : __ffs(~m) - 1;
      len += more;
      if (more < 32) break;
    }
    if (lane == 0) s_len[r] = len;
  }
  __syncthreads();
  const int heads = (int)p.c.heads, H2 = 2 * heads;
  const int sub = lane / LPR, ch = (lane % LPR) * 8;

  // an item by `nw` warps (1 or all), of which this is warp w
  auto item = [&](int r, int hh, int w, int nw) {
    const int t = s_run[r], len = s_len[r], which = hh / heads, h = hh % heads;
    const int slot = __ldg(p.slots + t), first = slot & (page - 1), pg = slot >> p.shift;
    const void* x = which ? p.x[1] : p.x[0];
    const int64_t ld = which ? p.ld[1] : p.ld[0], src = (int64_t)t * ld + (int64_t)h * DH + ch;
    float* scale_at = (which ? p.c.v_scale : p.c.k_scale) + (int64_t)pg * p.c.heads + h;
    uint8_t* dst = reinterpret_cast<uint8_t*>(which ? p.c.v : p.c.k) + (((int64_t)pg * p.c.heads + h) << p.shift) * DH + ch;
    const float present = first ? *scale_at : 0.f;
    Row8<BF16> row[IT];
    auto load = [&](int i0) {
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        const int i = i0 + q * RPP + sub;
        if (i < len) row[q].load(x, src + (int64_t)i * ld);
      }
    };
    uint32_t amax = 0;  // magnitudes order like their bits, NaN above all (bf16: two maxima side by side)
    for (int i0 = w * ROWS; i0 < len; i0 += nw * ROWS) {
      load(i0);
#pragma unroll
      for (int q = 0; q < IT; ++q)
        if (i0 + q * RPP + sub < len) row[q].amax(amax);
    }
    if constexpr (BF16) amax = max(amax & 0xffffu, amax >> 16) << 16;
    amax = __reduce_max_sync(0xffffffffu, amax);
    if (nw > 1) {
      if (lane == 0) s_amax[w] = amax;
      __syncthreads();  // everybody has read the present scale, too
#pragma unroll
      for (int k = 0; k < kWriteW; ++k) amax = max(amax, s_amax[k]);
    }
    const bool lost = amax >= 0x7f800000u || present != present;  // no scale holds these rows
    float s;
    if (lost) {
      s = __uint_as_float(0x7fc00000u);
    } else {
      s = pow2_scale<E4M3>(amax);
      if (first && present > s) s = present;
    }
    if (first && !lost && s != present) {
      // the scale grew: the page's older rows, rounded again
      const float f = __fdiv_rn(present, s);
      for (int i = w * RPP + sub; i < first; i += nw * RPP) {
        uint2 v = *reinterpret_cast<const uint2*>(dst + i * DH);
        float a[4], b[4];
        unpack4<E4M3>(v.x, a);
        unpack4<E4M3>(v.y, b);
        v.x = pack4<E4M3>(a[0] * f, a[1] * f, a[2] * f, a[3] * f);
        v.y = pack4<E4M3>(b[0] * f, b[1] * f, b[2] * f, b[3] * f);
        *reinterpret_cast<uint2*>(dst + i * DH) = v;
      }
    }
    const float inv = lost ? 0.f : __fdiv_rn(1.f, s);
    const bool again = len > nw * ROWS;
    for (int i0 = w * ROWS; i0 < len; i0 += nw * ROWS) {
      if (again) load(i0);
#pragma unroll
      for (int q = 0; q < IT; ++q) {
        const int i = i0 + q * RPP + sub;
        if (i < len) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = row[q].get(e) * inv;
          const uint2 bytes = make_uint2(pack4<E4M3>(v[0], v[1], v[2], v[3]), pack4<E4M3>(v[4], v[5], v[6], v[7]));
          *reinterpret_cast<uint2*>(dst + (first + i) * DH) = lost ? make_uint2(0, 0) : bytes;
        }
      }
    }
    if (w == 0 && lane == 0 && (first == 0 || s != present)) *scale_at = s;
    if (nw > 1) __syncthreads();  // s_amax is free again
    if (const uint32_t limit = byte_limit<E4M3>(s)) {
      __syncwarp();
      limit_rows<E4M3, DH>(dst, (s == present ? first : 0) + w * RPP + sub, nw * RPP, first + len, limit);
    }
  };

  for (int it = blockIdx.y * kWriteW + warp; it < s_n * H2; it += gridDim.y * kWriteW)
    if (s_len[it / H2] <= ROWS) item(it / H2, it % H2, 0, 1);
  for (int it = blockIdx.y; it < s_n * H2; it += gridDim.y)
    if (s_len[it / H2] > ROWS) item(it / H2, it % H2, warp, kWriteW);
}

// ------------------------------------------------------------------------------------
// kv8_read
// ------------------------------------------------------------------------------------

struct ReadParams {
  kv8_cache_t c;
  const int32_t* slots;
  void* out[2];
  int T, shift;
  int per_token, log_head;  // pieces of a token's row, and (as a shift) of a head's
  int32_t* status;
};

constexpr int kReadT = 256;  // threads per CTA
constexpr int kReadU = 4;    // pieces of a thread, their loads in flight together

// A piece is 16 bytes of the output: 8 channels (bf16) or 4 (float32), so that a warp's stores
// are whole lines; its 8 (4) bytes are loaded likewise. A CTA takes kReadT * kReadU consecutive
// pieces of the rows of one side. HBM-bound.
template <bool BF16, bool E4M3>
__global__ void __launch_bounds__(kReadT) k_kv8_read(ReadParams p) {
  constexpr int VEC = BF16 ? 8 : 4;
  const int64_t limit = p.c.n_pages << p.shift;
  const bool which = blockIdx.y != 0;
  const uint8_t* src = reinterpret_cast<const uint8_t*>(which ? p.c.v : p.c.k);
  const float* scales = which ? p.c.v_scale : p.c.k_scale;
  void* const out = which ? p.out[1] : p.out[0];
  if (!out) return;
  // the first piece's token, once per CTA; the rest by 32-bit arithmetic
  const int64_t first = (int64_t)blockIdx.x * (kReadT * kReadU);
  const int64_t t0 = first / p.per_token;
  const unsigned in0 = (unsigned)(first - t0 * p.per_token) + threadIdx.x;
  uint2 w[kReadU];
  float sc[kReadU];
  bool live[kReadU];
#pragma unroll
  for (int u = 0; u < kReadU; ++u) {
    const unsigned i = in0 + u * kReadT, dt = i / (unsigned)p.per_token, j = i - dt * (unsigned)p.per_token;
    const int64_t t = t0 + dt;
    w[u] = make_uint2(0, 0);
    sc[u] = 0.f;
    live[u] = t < p.T;
    if (live[u]) {
      const int s = __ldg(p.slots + t);
      if (s >= 0 && s < limit) {
        const int64_t head = (int64_t)(s >> p.shift) * p.c.heads + (j >> p.log_head);
        const uint8_t* at = src + ((head << p.shift) + (s & ((1 << p.shift) - 1))) * p.c.dh + (j & ((1u << p.log_head) - 1)) * VEC;
        if constexpr (BF16) w[u] = __ldg(reinterpret_cast<const uint2*>(at));
        else w[u].x = __ldg(reinterpret_cast<const uint32_t*>(at));
        sc[u] = __ldg(scales + head);
      } else if (s >= limit) {
        record_status(p.status, WINA_ERR_INVALID_ARG);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kReadU; ++u) {
    if (!live[u]) continue;
    uint4* d = reinterpret_cast<uint4*>(out) + first + threadIdx.x + u * kReadT;
    float a[4];
    unpack4<E4M3>(w[u].x, a);
    if constexpr (BF16) {
      float b[4];
      unpack4<E4M3>(w[u].y, b);
      uint32_t o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* f = e < 2 ? a : b;
        const __nv_bfloat162 x = __floats2bfloat162_rn(f[(2 * e) & 3] * sc[u], f[(2 * e + 1) & 3] * sc[u]);
        o[e] = *reinterpret_cast<const uint32_t*>(&x);
      }
      *d = make_uint4(o[0], o[1], o[2], o[3]);
    } else {
      *d = make_uint4(__float_as_uint(a[0] * sc[u]), __float_as_uint(a[1] * sc[u]), __float_as_uint(a[2] * sc[u]), __float_as_uint(a[3] * sc[u]));
    }
  }
}

static int page_shift(int64_t page) { return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7; }

static bool page_ok(int64_t page) { return page == 16 || page == 32 || page == 64 || page == kMaxPage; }

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

template <bool BF16, bool E4M3, int DH>
static void (*write_kernel(int64_t page))(WriteParams) {
  constexpr int ROWS = (BF16 ? 8 : 4) * (32 / (DH / 8));  // rows that a warp holds
  if constexpr (kMaxPage > 4 * ROWS)  // (bf16 rows of 64: no page is that long)
    if (page > 4 * ROWS) return k_kv8_write_shared<BF16, E4M3, DH>;
  return k_kv8_write<BF16, E4M3, DH>;
}

template <bool BF16, bool E4M3>
static void (*write_kernel(int64_t dh, int64_t page))(WriteParams) {
  return dh == 64 ? write_kernel<BF16, E4M3, 64>(page)
                  : dh == 128 ? write_kernel<BF16, E4M3, 128>(page) : write_kernel<BF16, E4M3, 256>(page);
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
  // the items of a stretch of tokens over several CTAs: eight at least, and more where few CTAs
  // would be running
  const int64_t gx = (T + p.seg - 1) / p.seg, most = 2 * cache->heads;
  const int64_t gy = std::min(most, std::max((most + kWriteW - 1) / kWriteW, (8 * sms + gx - 1) / gx));
  const bool e4 = cache->format == KV8_E4M3;
  void (*kern)(WriteParams) = xdt == WINA_BF16 ? (e4 ? write_kernel<true, true>(cache->dh, cache->page) : write_kernel<true, false>(cache->dh, cache->page))
                                               : (e4 ? write_kernel<false, true>(cache->dh, cache->page) : write_kernel<false, false>(cache->dh, cache->page));
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
  p.T = (int)T;
  const int vec = xdt == WINA_BF16 ? 8 : 4;
  p.per_token = (int)(cache->heads * cache->dh / vec);
  p.log_head = (cache->dh == 64 ? 6 : cache->dh == 128 ? 7 : 8) - (vec == 8 ? 3 : 2);
  p.shift = page_shift(cache->page);
  p.status = status_dev;
  const int64_t blocks = (T * p.per_token + kReadT * kReadU - 1) / (kReadT * kReadU);
  if (blocks > INT32_MAX) return WINA_ERR_INVALID_ARG;
  const dim3 grid((unsigned)blocks, 2);
  const bool e4 = cache->format == KV8_E4M3;
  void (*kern)(ReadParams) = xdt == WINA_BF16 ? (e4 ? k_kv8_read<true, true> : k_kv8_read<true, false>)
                                              : (e4 ? k_kv8_read<false, true> : k_kv8_read<false, false>);
  kern<<<grid, kReadT, 0, (cudaStream_t)stream>>>(p);
  return cuda_status(cudaGetLastError());
}
