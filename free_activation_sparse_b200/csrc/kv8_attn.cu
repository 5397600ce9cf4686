// Causal attention over the 8-bit paged key/value cache (kv8_attention).
//
//   s_j = (q . k8_j) ks[page_j] scale;  out = sum_j p_j vs[page_j] v8_j / sum_j p_j,
//   p_j = exp(s_j - max)
//
// k_kv8_attn_split: single tokens, short spans, and float32 prompts. Bound by HBM: every key
// and value byte is read once per block of 8 or 16 query rows (the rows of a kv head's query
// group, so grouped queries share the read).
#include <math.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "kv8.cuh"

namespace wina {

using namespace kv8;

constexpr float kLog2e = 1.4426950408889634f;

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
  uint32_t* counters;  // [kGridCap], zero between calls
  float* slots;        // [2 * kGridCap][slot_floats]
  int slot_floats;
  int stages;          // ring depth of k_kv8_attn_split
};

// ------------------------------------------------------------------------------------
// the work: tiles of query rows, chunks of keys
// ------------------------------------------------------------------------------------

// A request's queries and keys, clamped to what the tables hold.
struct Req {
  int q0, n, nq, kv;  // first row, queries, queries written (at most max_q), keys
};

__device__ __forceinline__ Req load_req(const AttnParams& p, int b) {
  Req r;
  if (p.cu_q) {
    const int a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
    r.q0 = max(0, min(a, p.T));
    r.n = max(0, min(e, p.T) - r.q0);
  } else {
    r.q0 = b;
    r.n = 1;
  }
  r.nq = min(r.n, p.max_q);
  const int room = p.width << p.shift;
  r.kv = max(0, min(__ldg(p.kv_len + b), room));
  return r;
}

// Whether load_req had to clamp something.
__device__ __forceinline__ bool bad_req(const AttnParams& p, int b) {
  bool bad = false;
  if (p.cu_q) {
    const int a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
    bad = a < 0 || e < a || e > p.T || e - a > p.max_q;
  }
  const int kv = __ldg(p.kv_len + b), room = p.width << p.shift;
  return bad || kv < 0 || kv > room;
}

// The keys [lo, hi) that rows r0 .. r0 + R - 1 of a request see (row = query * G + head in
// the group), and the chunks of CH keys they lie in. A tile that sees nothing has one chunk
// with no keys, so that its rows get their zeros on the common path.
struct Span {
  int lo, hi, c0, c1;
};

template <int R, int CH>
__device__ __forceinline__ Span tile_span(const AttnParams& p, const Req& r, int tile) {
  const int r0 = tile * R, r1 = min(r0 + R, r.nq * p.G) - 1;
  Span s;
  s.hi = r.kv - r.n + r1 / p.G + 1;
  s.lo = p.window > 0 ? max(0, r.kv - r.n + r0 / p.G - p.window + 1) : 0;
  if (s.hi <= s.lo) {
    s.lo = s.hi = s.c0 = 0;
    s.c1 = 1;
  } else {
    s.c0 = s.lo / CH;
    s.c1 = (s.hi + CH - 1) / CH;
  }
  return s;
}

template <int R>
__device__ __forceinline__ int tiles_of(const AttnParams& p, const Req& r) {
  return (r.nq * p.G + R - 1) / R;
}

// Chunks of all of a request's tiles, for one kv head.
template <int R, int CH>
__device__ __forceinline__ unsigned long long req_cost(const AttnParams& p, const Req& r) {
  const int nt = tiles_of<R>(p, r);
  unsigned long long c = 0;
  for (int t = 0; t < nt; ++t) {
    const Span s = tile_span<R, CH>(p, r, t);
    c += s.c1 - s.c0;
  }
  return c;
}

// Prefix sums over the requests of req_cost, in shared memory (pre[B] the total). Returns
// false where they pass 32 bits (more than 2^37 keys read: no cache is that large).
template <int NTHR, int R, int CH>
__device__ bool cost_prefix(const AttnParams& p, uint32_t* pre, uint32_t* red) {
  unsigned long long run = 0;
  __shared__ int s_over;
  if (threadIdx.x == 0) s_over = 0;
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += NTHR) {
    const int b = b0 + threadIdx.x;
    unsigned long long c = 0;
    if (b < p.B) {
      c = req_cost<R, CH>(p, load_req(p, b));
      if (blockIdx.x == 0 && bad_req(p, b)) record_status(p.status, WINA_ERR_INVALID_ARG);
    }
    if (c > 0xffffffffu / NTHR) s_over = 1;  // then the block's sum fits 32 bits below
    uint32_t total;
    const uint32_t ex = block_excl_scan<NTHR>((uint32_t)min(c, (unsigned long long)(0xffffffffu / NTHR)), red, &total);
    if (b < p.B) pre[b] = (uint32_t)run + ex;
    run += total;
    if (run > 0xffffffffu) s_over = 1;
  }
  if (threadIdx.x == 0) pre[p.B] = (uint32_t)run;
  __syncthreads();
  return s_over == 0;
}

// A walk over tiles: requests in order, in each the kv heads, in each the row tiles.
template <int R, int CH>
struct Walk {
  int b, hk, tile, nt;
  Req r;
  Span s;
  unsigned long long at;  // chunks before this tile, over all heads

  __device__ __forceinline__ void locate(const AttnParams& p, const uint32_t* pre, unsigned long long u) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned long long)pre[mid] * p.c.heads <= u) lo = mid;
      else hi = mid;
    }
    b = lo;
    r = load_req(p, b);
    nt = tiles_of<R>(p, r);
    const unsigned cost = pre[b + 1] - pre[b];
    const unsigned long long rem = u - (unsigned long long)pre[b] * p.c.heads;
    hk = (int)(rem / cost);
    unsigned in = (unsigned)(rem - (unsigned long long)hk * cost);
    tile = 0;
    s = tile_span<R, CH>(p, r, 0);
    while (in >= (unsigned)(s.c1 - s.c0)) {
      in -= s.c1 - s.c0;
      s = tile_span<R, CH>(p, r, ++tile);
    }
    at = u - in;
  }
  // to the next tile (there is one)
  __device__ __forceinline__ void next(const AttnParams& p, const uint32_t* pre) {
    at += s.c1 - s.c0;
    if (++tile == nt) {
      tile = 0;
      if (++hk == (int)p.c.heads) {
        hk = 0;
        do ++b;
        while (b < p.B - 1 && pre[b + 1] == pre[b]);
        r = load_req(p, b);
        nt = tiles_of<R>(p, r);
      }
    }
    s = tile_span<R, CH>(p, r, tile);
  }
};

// The work's [0, C) chunks over nc teams: team i has [C i / nc, C (i + 1) / nc); the team
// that has chunk u.
__device__ __forceinline__ unsigned long long team_start(unsigned long long C, int nc, int i) { return C * i / nc; }
__device__ __forceinline__ int team_of(unsigned long long C, int nc, unsigned long long u) {
  return (int)(((u + 1) * nc - 1) / C);
}

// ------------------------------------------------------------------------------------
// k_kv8_attn_split
// ------------------------------------------------------------------------------------

constexpr int kSplitW = 8;                  // warps per CTA
constexpr int kSplitT = 32 * kSplitW;
constexpr int kMergeBytes = 16 * 1024;      // merge buffer of a CTA
constexpr float kPScaleLog2 = 14.f;         // weights are held times 2^14 (float16's middle)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// D += A B, 16 x 8 x 16, float16 operands, float32 accumulators.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit elements spread over a warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The two low (high) bytes of w as float16 numbers. Exact: int8 through 1024 + (byte + 128),
// whose float16 step is 1; e4m3 is a subset of float16. `biased`: an int8 word already
// xor-ed with 0x80808080.
template <bool E4M3, bool HIGH>
__device__ __forceinline__ uint32_t half2_of(uint32_t w) {
  if constexpr (E4M3) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(HIGH ? w >> 16 : w & 0xffffu), __NV_E4M3);
    return (uint32_t)h.x | ((uint32_t)h.y << 16);
  } else {
    const uint32_t u = __byte_perm(w, 0x64646464u, HIGH ? 0x4342 : 0x4140);
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}
template <bool E4M3>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
  return E4M3 ? w : w ^ 0x80808080u;
}

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte piece c of row r in a staged tile of DH-byte rows: the pieces are
// permuted so that both the key reads (8 lanes: 2 rows, 4 pieces) and the value reads (8
// lanes: 4 rows, 2 pieces) fall on different banks.
template <int DH>
__device__ __forceinline__ uint32_t staged(int r, int c) {
  if constexpr (DH == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return r * DH + ((c ^ (r & 7)) << 4);
}

// One CTA of eight warps per SM. The work (tiles of 8 NT query rows of one request and kv
// head, times the chunks of CH keys they see) is a line cut into equal parts, one per CTA,
// so that one long sequence fills the GPU and a ragged batch is balanced; a CTA's chunks of
// one tile go round its warps. Each warp has its own ring of `stages` chunks, filled with
// cp.async (keys, values and the pages' scales; places outside the tile's keys are filled
// with zeros and never read), and runs on across tiles, so loads stay in flight while tiles
// are joined.
//
// Per chunk, with keys as the rows of the matrix instruction, so that 8 query rows cost half
// of what 16 do:
//   S^T = K Q^T   bytes to float16 (exact), queries as float16 times a power of two per row
//                 (bf16: exact; float32: two float16 parts, 2^-22 of the row's largest), the
//                 channels in the order the 16-byte reads deliver them, which the sum does
//                 not mind;
//   running max, p = 2^(s - max + 14), sum p in float32;
//   O^T += V^T P^T with P = p vs / sref in float16 (float32: two parts), sref the largest
//                 value scale met so far: a weight keeps 11 (22) bits down to 2^-28 of the
//                 largest, and O is rescaled where max or sref grow.
// The eight warps' (max, sum, O) are joined in shared memory in warp order; a tile cut by a
// part's end is left in the workspace, and the last CTA of that tile to arrive joins the
// parts in order. No CTA waits for another.
template <bool BF16, bool E4M3, int DH, int NT>
__global__ void __launch_bounds__(kSplitT, 1) k_kv8_attn_split(AttnParams p) {
  constexpr int CH = DH == 256 ? 16 : 32;     // keys of a chunk
  constexpr int MT = CH / 16;                 // 16-key groups of a chunk
  constexpr int R = 8 * NT;                   // query rows of a tile
  constexpr int KS = DH / 16;                 // k-steps of a score, and 16-channel tiles of O
  constexpr int KC = DH / 64;                 // 16-byte pieces of a key row per lane
  constexpr int PARTS = BF16 ? 1 : 2;
  constexpr int STAGE = 2 * CH * DH;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint32_t red[32];
  __shared__ float s_m[kSplitW][R], s_l[kSplitW][R];
  __shared__ float s_meta[kSplitW][3][4];     // ks, vs of a chunk's 16-key groups
  __shared__ uint32_t s_bad[kSplitW][3];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int S = p.stages;
  unsigned char* ring = sm + (size_t)warp * S * STAGE;
  float* mbuf = reinterpret_cast<float*>(sm + (size_t)kSplitW * S * STAGE);
  uint32_t* pre = reinterpret_cast<uint32_t*>(sm + (size_t)kSplitW * S * STAGE + kMergeBytes);
  if (!cost_prefix<kSplitT, R, CH>(p, pre, red)) {
    if (blockIdx.x == 0 && tid == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
    return;
  }
  const unsigned long long C = (unsigned long long)pre[p.B] * p.c.heads;
  if (C == 0) return;
  // at least one chunk for each warp of a team
  const int nc = (int)min((unsigned long long)gridDim.x, (C + kSplitW - 1) / kSplitW);
  if ((int)blockIdx.x >= nc) return;
  const unsigned long long u0 = team_start(C, nc, blockIdx.x), u1 = team_start(C, nc, blockIdx.x + 1);

  using W = Walk<R, CH>;
  W cons, prod;  // the tile being computed, the tile being loaded
  cons.locate(p, pre, u0);
  prod = cons;
  // the chunks [from, to) of a tile that this CTA has; this warp's are from + warp, + 8, ...
  auto part = [&](const W& w, int& from, int& to) {
    from = w.s.c0 + (int)(u0 > w.at ? u0 - w.at : 0);
    const unsigned long long end = w.at + (unsigned)(w.s.c1 - w.s.c0);
    to = end > u1 ? w.s.c1 - (int)(end - u1) : w.s.c1;
  };
  int pc, pto;  // the producer's next chunk
  part(prod, pc, pto);
  pc += warp;
  bool more = true;
  // page indices of the producer's next chunks, one chunk to a lane
  int pg0 = -1, pg1 = -1, pg_from = -1, pg_b = -1;

  const int page_mask = (1 << p.shift) - 1;
  // issue the next chunk of this warp into `stage`
  auto issue = [&](int stage) {
    while (more && pc >= pto) {  // the next tile with a chunk for this warp
      if (prod.at + (unsigned)(prod.s.c1 - prod.s.c0) >= u1) {
        more = false;
        break;
      }
      prod.next(p, pre);
      part(prod, pc, pto);
      pc += warp;
    }
    if (more) {
      const int off = pc - pg_from;
      if (pg_b != prod.b || off < 0 || off >= 32 * kSplitW || (off & (kSplitW - 1))) {
        pg_b = prod.b;
        pg_from = pc;
        const int64_t key = (int64_t)(pc + lane * kSplitW) * CH;
        const int32_t* row = p.table + (int64_t)prod.b * p.width;
        pg0 = key < prod.r.kv ? __ldg(row + (key >> p.shift)) : -1;
        if (MT == 2) pg1 = key + 16 < prod.r.kv ? __ldg(row + ((key + 16) >> p.shift)) : -1;
      }
      const int from = (pc - pg_from) / kSplitW;
      const int key0 = pc * CH;
      int64_t head[MT];  // (page, head) of each 16-key group, in rows of the cache
      uint32_t bad = 0;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const int pg = __shfl_sync(0xffffffffu, u ? pg1 : pg0, from);
        const bool used = key0 + 16 * u < prod.s.hi && key0 + 16 * u + 16 > prod.s.lo;
        const bool ok = used && pg >= 0 && pg < p.c.n_pages;
        head[u] = ok ? (int64_t)pg * p.c.heads + prod.hk : -1;
        if (used && !ok) {
          bad |= 1u << u;
          if (lane == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
        }
      }
      const uint32_t dst = (uint32_t)__cvta_generic_to_shared(ring + (size_t)stage * STAGE);
      constexpr int PPR = DH / 16;  // pieces per row
#pragma unroll
      for (int i = 0; i < CH * PPR / 32; ++i) {
        const int piece = i * 32 + lane, row = piece / PPR, c = piece % PPR, key = key0 + row;
        const int64_t h = head[MT == 2 ? (i * 32 / PPR) / 16 : 0];  // a pass stays in one group
        const bool on = h >= 0 && key >= prod.s.lo && key < prod.s.hi;
        const int64_t src = on ? ((h << p.shift) + (key & page_mask)) * DH + c * 16 : 0;
        const uint32_t d = dst + staged<DH>(row, c);
        cp_async16(d, reinterpret_cast<const uint8_t*>(p.c.k) + src, on ? 16 : 0);
        cp_async16(d + CH * DH, reinterpret_cast<const uint8_t*>(p.c.v) + src, on ? 16 : 0);
      }
      if (lane < 2 * MT) {
        const int64_t h = (MT == 2 && (lane & 1)) ? head[MT - 1] : head[0];
        const float* s = (lane >= MT ? p.c.v_scale : p.c.k_scale) + (h >= 0 ? h : 0);
        cp_async4((uint32_t)__cvta_generic_to_shared(&s_meta[warp][stage][lane]), s, h >= 0 ? 4 : 0);
      }
      if (lane == 0) s_bad[warp][stage] = bad;
      pc += kSplitW;
    }
    cp_commit();
  };

  for (int i = 0; i < S - 1; ++i) issue(i);
  int stage = 0;

  for (;;) {  // tiles
    int from, to;
    part(cons, from, to);
    const int rows = min(R, cons.r.nq * p.G - cons.tile * R);
    // queries: lane (g, t) has row g's pieces of channels as the keys' lanes t have them
    uint32_t qf[PARTS][NT][KS][2];
    float cr[NT][2];  // factor of a score, rows 2t and 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g, rr = cons.tile * R + row;
      const int64_t at = (int64_t)(cons.r.q0 + rr / p.G) * p.ld_q + (int64_t)(cons.hk * p.G + rr % p.G) * DH;
      float f[KC][16], big = 0.f;
#pragma unroll
      for (int j = 0; j < KC; ++j) {
        const int c = DH == 64 ? t : (j >> 1) * 8 + 2 * t + (j & 1);
        Row8<BF16> a, b;
        if (row < rows) {
          a.load(p.q, at + c * 16);
          b.load(p.q, at + c * 16 + 8);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[j][e] = row < rows ? a.get(e) : 0.f;
          f[j][8 + e] = row < rows ? b.get(e) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) big = fmaxf(big, fabsf(f[j][e]));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the row's largest number goes to [2^14, 2^15)
      int ex = (int)(__float_as_uint(big) >> 23);
      ex = ex == 255 ? 127 : max(15, ex);  // infinities and NaN stay what they are
      const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);
      const float dn = __fdiv_rn(1.f, up);
#pragma unroll
      for (int j = 0; j < KC; ++j)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = f[j][4 * w + 2 * e] * up, y = f[j][4 * w + 2 * e + 1] * up;
            const __half2 h = __floats2half2_rn(x, y);
            qf[0][nt][j * 4 + w][e] = *reinterpret_cast<const uint32_t*>(&h);
            if constexpr (!BF16) {
              const float2 back = __half22float2(h);
              qf[PARTS - 1][nt][j * 4 + w][e] = pack_half2(x - back.x, y - back.y);
            }
          }
      const float fac = dn * p.scale * (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
      cr[nt][0] = __shfl_sync(0xffffffffu, fac, 8 * t);
      cr[nt][1] = __shfl_sync(0xffffffffu, fac, 8 * t + 4);
    }
    // rows 2t, 2t + 1 (+ 8): the keys they see
    int lim[NT][2], low[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = cons.tile * R + min(nt * 8 + 2 * t + e, rows - 1);
        lim[nt][e] = cons.r.kv - cons.r.n + rr / p.G + 1;
        low[nt][e] = p.window > 0 ? lim[nt][e] - p.window : 0;
      }
    // chunks between these need no masks
    const int first_lim = cons.r.kv - cons.r.n + cons.tile * R / p.G + 1;
    const int last_low = p.window > 0 ? cons.r.kv - cons.r.n + (cons.tile * R + rows - 1) / p.G + 1 - p.window : 0;

    float o[NT][KS][4], m[NT][2], l[NT][2], sref = 1.17549435e-38f, inv_sref = 1.f / 1.17549435e-38f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < KS; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][j][e] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    for (int c = from + warp; c < to; c += kSplitW) {
      if (S == 3) cp_wait<1>();
      else cp_wait<0>();
      __syncwarp();
      issue(stage == 0 ? S - 1 : stage - 1);
      const unsigned char* kst = ring + (size_t)stage * STAGE;
      const unsigned char* vst = kst + CH * DH;
      float s[NT][MT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][u][e] = 0.f;
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const int cc = DH == 64 ? t : (j >> 1) * 8 + 2 * t + (j & 1);
          const uint4 x = *reinterpret_cast<const uint4*>(kst + staged<DH>(u * 16 + g, cc));
          const uint4 y = *reinterpret_cast<const uint4*>(kst + staged<DH>(u * 16 + g + 8, cc));
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t a = biased<E4M3>(xs[w]), b = biased<E4M3>(ys[w]);
            const uint32_t fr[4] = {half2_of<E4M3, false>(a), half2_of<E4M3, false>(b), half2_of<E4M3, true>(a),
                                    half2_of<E4M3, true>(b)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < PARTS; ++q) mma16816(s[nt][u], fr, qf[q][nt][j * 4 + w][0], qf[q][nt][j * 4 + w][1]);
          }
        }
      float ks[MT], vs[MT];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        ks[u] = s_meta[warp][stage][u];
        vs[u] = s_meta[warp][stage][MT + u];
      }
      const uint32_t bad = s_bad[warp][stage];
      const int key0 = c * CH;
      const bool masked = bad || key0 < last_low || key0 < cons.s.lo || key0 + CH > first_lim;
      // scores in units of log 2
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = s[nt][u][e] * (cr[nt][e & 1] * ks[u]);
            if (p.softcap > 0.f) x = tanhf(x) * (p.softcap * kLog2e);
            s[nt][u][e] = x;
          }
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < MT; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = key0 + 16 * u + g + (e >> 1) * 8;
              if (key >= lim[nt][e & 1] || key < low[nt][e & 1] || ((bad >> u) & 1)) s[nt][u][e] = -INFINITY;
            }
      }
      bool grew = false;
      float mb[NT][2], al[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[nt][0][e], s[nt][0][e + 2]);
          if (MT == 2) x = fmaxf(x, fmaxf(s[nt][MT - 1][e], s[nt][MT - 1][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          x = fmaxf(x, m[nt][e]);
          grew |= x > m[nt][e];
          al[nt][e] = x > m[nt][e] ? ex2(m[nt][e] - x) : 1.f;
          m[nt][e] = x;
          mb[nt][e] = x == -INFINITY ? 0.f : x - kPScaleLog2;
        }
      float vmax = sref;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const float a = fabsf(vs[u]);
        if (a < INFINITY && !((bad >> u) & 1)) vmax = fmaxf(vmax, a);
      }
      if (__any_sync(0xffffffffu, grew) || vmax > sref) {
        const float down = sref * __fdiv_rn(1.f, vmax);
        sref = vmax;
        inv_sref = __fdiv_rn(1.f, vmax);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][j][e] *= al[nt][e & 1] * down;
          l[nt][0] *= al[nt][0];
          l[nt][1] *= al[nt][1];
        }
      }
      uint32_t pf[PARTS][NT][MT][2];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const float ratio = vs[u] * inv_sref;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = ex2(s[nt][u][e] - mb[nt][e & 1]);
            l[nt][e & 1] += w[e];
            // a weight of 0 stays 0 under any scale
            w[e] = w[e] == 0.f ? 0.f : w[e] * ratio;
          }
          const __half2 a = __floats2half2_rn(w[0], w[1]), b = __floats2half2_rn(w[2], w[3]);
          pf[0][nt][u][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&a));
          pf[0][nt][u][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&b));
          if constexpr (!BF16) {
            const float2 fa = __half22float2(a), fb = __half22float2(b);
            pf[PARTS - 1][nt][u][0] = transpose8x8(pack_half2(w[0] - fa.x, w[1] - fa.y));
            pf[PARTS - 1][nt][u][1] = transpose8x8(pack_half2(w[2] - fb.x, w[3] - fb.y));
          }
        }
      }
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int h = 0; h < (DH == 256 ? 2 : 1); ++h) {
          constexpr int VW = DH == 64 ? 2 : 4;  // words of a key's channels per lane
          uint32_t x[4][VW];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = u * 16 + 2 * t + (k & 1) + (k >> 1) * 8;
            if constexpr (DH == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(vst + staged<DH>(row, g >> 1) + (g & 1) * 8);
              x[k][0] = biased<E4M3>(v.x);
              x[k][1] = biased<E4M3>(v.y);
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(vst + staged<DH>(row, h * 8 + g));
              x[k][0] = biased<E4M3>(v.x);
              x[k][1] = biased<E4M3>(v.y);
              x[k][2] = biased<E4M3>(v.z);
              x[k][3] = biased<E4M3>(v.w);
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            // channels 4w, 4w + 1 of two keys side by side, then 4w + 2, 4w + 3
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a = __byte_perm(x[0][w], x[1][w], e ? 0x7362 : 0x5140);
              const uint32_t b = __byte_perm(x[2][w], x[3][w], e ? 0x7362 : 0x5140);
              const uint32_t fr[4] = {half2_of<E4M3, false>(a), half2_of<E4M3, true>(a), half2_of<E4M3, false>(b),
                                      half2_of<E4M3, true>(b)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int q = 0; q < PARTS; ++q)
                  mma16816(o[nt][h * 8 + 2 * w + e], fr, pf[q][nt][u][0], pf[q][nt][u][1]);
            }
          }
        }
      stage = stage == S - 1 ? 0 : stage + 1;
    }

    // ---- join the warps' parts of this tile ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t + e] = m[nt][e];
          s_l[warp][nt * 8 + 2 * t + e] = x;
        }
      }
    __syncthreads();
    const bool whole = from == cons.s.c0 && to == cons.s.c1;
    // this CTA's slot: a part that begins its tile elsewhere comes first
    float* slot = p.slots + (size_t)(2 * blockIdx.x + (from == cons.s.c0 ? 1 : 0)) * p.slot_floats;
    float fac[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t + e;
        float M = -INFINITY;
        for (int w = 0; w < kSplitW; ++w) M = fmaxf(M, s_m[w][row]);
        fac[nt][e] = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - M) * sref;
      }
    // rounds of RC channels of 8 rows
    constexpr int RC = kMergeBytes / (kSplitW * 8 * 4) < DH ? kMergeBytes / (kSplitW * 8 * 4) : DH;
    constexpr int CPL = DH == 64 ? 8 : 16;  // consecutive channels a lane has of a 128-channel half
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += RC) {
        // lane (g, t): rows 2t, 2t + 1, channels g * CPL .. (+ 128 for the second half)
#pragma unroll
        for (int h = 0; h < (DH == 256 ? 2 : 1); ++h) {
          const int ch = h * 128 + g * CPL;
          if (ch >= c0 && ch < c0 + RC) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float* d = mbuf + ((size_t)warp * 8 + 2 * t + e) * RC + (ch - c0);
#pragma unroll
              for (int q = 0; q < CPL / 4; ++q)
                *reinterpret_cast<float4*>(d + 4 * q) =
                    make_float4(o[nt][h * 8 + 2 * q][e] * fac[nt][e], o[nt][h * 8 + 2 * q][e + 2] * fac[nt][e],
                                o[nt][h * 8 + 2 * q + 1][e] * fac[nt][e], o[nt][h * 8 + 2 * q + 1][e + 2] * fac[nt][e]);
            }
          }
        }
        __syncthreads();
        for (int i = tid; i < 8 * RC / 4; i += kSplitT) {
          const int row = i / (RC / 4), ch = (i % (RC / 4)) * 4, rr = nt * 8 + row;
          if (rr >= rows) continue;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kSplitW; ++w) {
            const float4 x = *reinterpret_cast<const float4*>(mbuf + ((size_t)w * 8 + row) * RC + ch);
            a.x += x.x;
            a.y += x.y;
            a.z += x.z;
            a.w += x.w;
          }
          if (whole) {
            float M = -INFINITY, L = 0.f;
            for (int w = 0; w < kSplitW; ++w) M = fmaxf(M, s_m[w][rr]);
            for (int w = 0; w < kSplitW; ++w) L += s_m[w][rr] == -INFINITY ? 0.f : s_l[w][rr] * ex2(s_m[w][rr] - M);
            const float inv = L == 0.f ? 0.f : 1.f / L;
            const int qr = cons.tile * R + rr;
            const int64_t at = ((int64_t)(cons.r.q0 + qr / p.G) * p.Hq + cons.hk * p.G + qr % p.G) * DH + c0 + ch;
            if constexpr (BF16) {
              const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
              *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
            } else {
              *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) =
                  make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
            }
          } else {
            *reinterpret_cast<float4*>(slot + (size_t)rr * DH + c0 + ch) = a;
          }
        }
        __syncthreads();
      }
    }
    if (!whole) {
      if (tid < rows) {
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < kSplitW; ++w) M = fmaxf(M, s_m[w][tid]);
        for (int w = 0; w < kSplitW; ++w) L += s_m[w][tid] == -INFINITY ? 0.f : s_l[w][tid] * ex2(s_m[w][tid] - M);
        slot[R * DH + tid] = M;
        slot[R * DH + R + tid] = L;
      }
      // the tile's parts lie with teams ta .. tb, the first of which names its counter
      const unsigned len = cons.s.c1 - cons.s.c0;
      const int ta = team_of(C, nc, cons.at), tb = team_of(C, nc, cons.at + len - 1), parts = tb - ta + 1;
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        s_last = atomicAdd(p.counters + ta, 1u) == (unsigned)(parts - 1);
        if (s_last) p.counters[ta] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        // team ta's part is the last of its line (slot 1), the others' the first of theirs
        auto part_of = [&](int i) { return p.slots + (size_t)(2 * (ta + i) + (i == 0 ? 1 : 0)) * p.slot_floats; };
        for (int i = tid; i < rows * DH / 4; i += kSplitT) {
          const int rr = i / (DH / 4), ch = (i % (DH / 4)) * 4;
          float M = -INFINITY;
          for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(part_of(k) + R * DH + rr));
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
          float L = 0.f;
          for (int k = 0; k < parts; ++k) {
            const float* q = part_of(k);
            const float mk = __ldcg(q + R * DH + rr), w = mk == -INFINITY ? 0.f : ex2(mk - M);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + (size_t)rr * DH + ch));
            L += __ldcg(q + R * DH + R + rr) * w;
            a.x += x.x * w;
            a.y += x.y * w;
            a.z += x.z * w;
            a.w += x.w * w;
          }
          const float inv = L == 0.f ? 0.f : 1.f / L;
          const int qr = cons.tile * R + rr;
          const int64_t at = ((int64_t)(cons.r.q0 + qr / p.G) * p.Hq + cons.hk * p.G + qr % p.G) * DH + ch;
          if constexpr (BF16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(a.x * inv, a.y * inv), y = __floats2bfloat162_rn(a.z * inv, a.w * inv);
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
          } else {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) =
                make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
          }
        }
      }
    }
    if (cons.at + (unsigned)(cons.s.c1 - cons.s.c0) >= u1) break;
    cons.next(p, pre);
    __syncthreads();  // s_m, s_l and the merge buffer are free again
  }
  cp_wait<0>();
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------

// Query rows of a tile of k_kv8_attn_split: 8 or 16 (8 where a row is 256 wide: 16 rows of
// sums would not fit the registers).
static int split_rows(int64_t dh, int64_t rows) { return rows <= 8 || dh == 256 ? 8 : 16; }

static size_t split_slot_floats(int64_t dh, int64_t rows) { return (size_t)split_rows(dh, rows) * (dh + 2); }

size_t kv8_attention_ws_size(int64_t dh, int64_t rows) {
  return round_up((size_t)kGridCap * 4, kAlign) + round_up((size_t)2 * kGridCap * split_slot_floats(dh, rows) * 4, kAlign);
}

template <bool BF16, bool E4M3>
static void (*split_kernel(int64_t dh, int rows))(AttnParams) {
  if (dh == 64) return rows == 8 ? k_kv8_attn_split<BF16, E4M3, 64, 1> : k_kv8_attn_split<BF16, E4M3, 64, 2>;
  if (dh == 128) return rows == 8 ? k_kv8_attn_split<BF16, E4M3, 128, 1> : k_kv8_attn_split<BF16, E4M3, 128, 2>;
  return k_kv8_attn_split<BF16, E4M3, 256, 1>;
}

static wina_status_t launch_split(AttnParams& p, bool bf16, int64_t rows, cudaStream_t s) {
  const int64_t dh = p.c.dh;
  const int R = split_rows(dh, rows);
  const size_t stage = (size_t)2 * (dh == 256 ? 16 : 32) * dh * kSplitW, pre = round_up((size_t)(p.B + 1) * 4, 16);
  // three chunks a warp, or two where a very large batch's prefix sums need the room
  p.stages = 3;
  size_t smem = 3 * stage + kMergeBytes + pre;
  if (smem > (size_t)222 * 1024) {
    p.stages = 2;
    smem -= stage;
  }
  p.slot_floats = (int)split_slot_floats(dh, rows);
  const bool e4 = p.c.format == KV8_E4M3;
  void (*kern)(AttnParams) = bf16 ? (e4 ? split_kernel<true, true>(dh, R) : split_kernel<true, false>(dh, R))
                                  : (e4 ? split_kernel<false, true>(dh, R) : split_kernel<false, false>(dh, R));
  const int sms = device_sm_count();
  if (sms < 1) return WINA_ERR_CUDA;
  return cuda_status(launch_kernel(kern, dim3((unsigned)std::min(sms, kGridCap)), dim3(kSplitT), smem, s, false, p));
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
      max_q < 1 || max_q > (1 << 24) || width < 1 || width > (1 << 30) / cache->page || window < 0 ||
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
  p.window = window >= width * cache->page ? 0 : (int)window;  // as wide as the table: no window
  p.out = out;
  p.status = status_dev;
  p.counters = reinterpret_cast<uint32_t*>(ws);
  p.slots = reinterpret_cast<float*>((char*)ws + round_up((size_t)kGridCap * 4, kAlign));
  return launch_split(p, qdt == WINA_BF16, max_q * (Hq / cache->heads), (cudaStream_t)stream);
}
