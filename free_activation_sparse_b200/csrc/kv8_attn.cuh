// What the attention kernels over the 8-bit paged cache share: their parameters, the line of
// work and the walks over it, and the conversions of bytes.
#pragma once

#include "internal.h"
#include "kv8.cuh"
#include "tc.cuh"

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
  uint32_t* counters;  // [kMaxTeams], zero between calls
  float* slots;        // [2 * kMaxTeams][slot_floats]
  int slot_floats;
  int tiles;      // tiles of query rows, over all heads, at most
  int tile_cost;  // a tile's fixed cost, in chunks
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

constexpr unsigned kEmptyCost = 4;

// The keys [lo, hi) that rows r0 .. r0 + R - 1 of a request see (row = query * G + head in
// the group), and the chunks of CH keys they lie in; none for a tile that sees nothing.
struct Span {
  int lo, hi, c0, c1;
  // Units on the line of work: the chunks, and what a tile costs besides (its queries, the
  // joining of its parts), p.tile_cost, before its first chunk; kEmptyCost where rows only get
  // zeros (in a request with keys; one without any is not on the line).
  __device__ __forceinline__ unsigned len(const AttnParams& p) const { return c1 > c0 ? (unsigned)(c1 - c0 + p.tile_cost) : kEmptyCost; }
};

template <int R, int CH>
__device__ __forceinline__ Span tile_span(const AttnParams& p, const Req& r, int tile) {
  const int r0 = tile * R, r1 = min(r0 + R, r.nq * p.G) - 1;
  Span s;
  s.hi = r.kv - r.n + r1 / p.G + 1;
  s.lo = p.window > 0 ? max(0, r.kv - r.n + r0 / p.G - p.window + 1) : 0;
  if (s.hi <= s.lo) {
    s.lo = s.hi = s.c0 = s.c1 = 0;
  } else {
    s.c0 = s.lo / CH;
    s.c1 = (s.hi + CH - 1) / CH;
  }
  return s;
}

template <int R>
__device__ __forceinline__ int tiles_of(const AttnParams& p, const Req& r) {
  return r.kv ? (r.nq * p.G + R - 1) / R : 0;
}

// Zeros for the requests without keys (a padded batch's places), dealt over the grid.
template <bool BF16>
__device__ __forceinline__ void zero_rows(const AttnParams& p) {
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    const Req r = load_req(p, b);
    if (r.kv) continue;
    const int64_t row = (int64_t)p.Hq * p.c.dh * (BF16 ? 2 : 4) / 16;  // 16-byte pieces of a query
    uint4* d = reinterpret_cast<uint4*>(p.out) + r.q0 * row;
    for (int64_t i = threadIdx.x; i < r.nq * row; i += blockDim.x) d[i] = make_uint4(0, 0, 0, 0);
  }
}

// Units of all of a request's tiles, for one kv head.
template <int R, int CH>
__device__ __forceinline__ unsigned long long req_cost(const AttnParams& p, const Req& r) {
  const int nt = tiles_of<R>(p, r);
  unsigned long long c = 0;
  for (int t = 0; t < nt; ++t) {
    c += tile_span<R, CH>(p, r, t).len(p);
  }
  return c;
}

// x + y, 2^32 - 1 where the sum passes 32 bits.
__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) {
  const uint32_t s = x + y;
  return s < x ? 0xffffffffu : s;
}

// block_excl_scan with sums that stay at 2^32 - 1 once they reach it (the prefixes then mean nothing).
template <int NTHR>
__device__ __forceinline__ uint32_t block_excl_scan_sat(uint32_t v, uint32_t* red, uint32_t* total) {
  constexpr int NW = NTHR / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = add_sat(x, y);
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t w = lane < NW ? red[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w = add_sat(w, y);
    }
    if (lane < NW) red[lane] = w;  // inclusive over warps
  }
  __syncthreads();
  const uint32_t before = warp ? red[warp - 1] : 0u;
  *total = red[NW - 1];
  __syncthreads();
  return before + x - v;
}

// Prefix sums of req_cost before every fourth request, in shared memory (pre[ceil(B / 4)] the
// total). Returns false for a call that no cache's attention needs and that would run for
// minutes to hours: 2^32 units or more for one kv head (the sums are 32 bits wide), or 2^36
// over all heads (so that a team's chunks can be counted in 31 bits).
constexpr int kPreStep = 4;
__host__ __device__ constexpr int pre_entries(int B) { return (B + kPreStep - 1) / kPreStep + 1; }

template <int NTHR, int R, int CH>
__device__ bool cost_prefix(const AttnParams& p, uint32_t* pre, uint32_t* red) {
  unsigned long long run = 0;  // the same in all threads
  bool fits = true;
  for (int b0 = 0; b0 < p.B; b0 += NTHR) {
    const int b = b0 + threadIdx.x;
    unsigned long long c = 0;
    if (b < p.B) {
      c = req_cost<R, CH>(p, load_req(p, b));
      if (blockIdx.x == 0 && bad_req(p, b)) record_status(p.status, WINA_ERR_INVALID_ARG);
    }
    uint32_t total;
    const uint32_t ex = block_excl_scan_sat<NTHR>((uint32_t)min(c, 0xffffffffull), red, &total);
    if (b < p.B && b % kPreStep == 0) pre[b / kPreStep] = (uint32_t)run + ex;
    run += total;
    fits = fits && total != 0xffffffffu;
  }
  if (threadIdx.x == 0) pre[pre_entries(p.B) - 1] = (uint32_t)run;
  __syncthreads();
  return fits && run <= 0xffffffffu && run * p.c.heads < (1ull << 36);
}

// A walk over tiles: requests in order, in each the kv heads, in each the row tiles.
template <int R, int CH>
struct Walk {
  int b, hk, tile, nt;
  Req r;
  Span s;
  unsigned long long at;  // the line's units before this tile

  __device__ __forceinline__ unsigned len(const AttnParams& p) const { return s.len(p); }
  // The chunks [from, to) of the tile that the team of units [u0, u1) has; none where its part of
  // the line ends in the tile's fixed cost, and none of a tile that sees no key, wherever the
  // part ends in it.
  __device__ __forceinline__ void part(const AttnParams& p, unsigned long long u0, unsigned long long u1, int& from, int& to) const {
    const unsigned long long first = at + p.tile_cost, end = at + len(p);
    from = s.c0 + (int)(u0 > first ? u0 - first : 0);
    to = u1 >= end ? s.c1 : u1 > first ? min(s.c1, s.c0 + (int)(u1 - first)) : s.c0;
  }
  // whether the tile's rows only get zeros, and the team of units [u0, u1) is to write them
  __device__ __forceinline__ bool empty_of(unsigned long long u0, unsigned long long u1) const {
    return s.c0 == s.c1 && at >= u0 && at < u1;
  }

  // the tile that holds unit u
  __device__ __forceinline__ void locate(const AttnParams& p, const uint32_t* pre, unsigned long long u) {
    int lo = 0, hi = pre_entries(p.B) - 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((unsigned long long)pre[mid] * p.c.heads <= u) lo = mid;
      else hi = mid;
    }
    b = lo * kPreStep;
    unsigned long long rem = u - (unsigned long long)pre[lo] * p.c.heads, cost;
    for (;; ++b) {
      r = load_req(p, b);
      cost = req_cost<R, CH>(p, r);
      if (rem < cost * p.c.heads) break;
      rem -= cost * p.c.heads;
    }
    nt = tiles_of<R>(p, r);
    hk = (int)(rem / cost);
    unsigned in = (unsigned)(rem - (unsigned long long)hk * cost);
    tile = 0;
    s = tile_span<R, CH>(p, r, 0);
    while (in >= len(p)) {
      in -= len(p);
      s = tile_span<R, CH>(p, r, ++tile);
    }
    at = u - in;
  }
  // to the next tile (there is one)
  __device__ __forceinline__ void next(const AttnParams& p) {
    at += len(p);
    if (++tile == nt) {
      tile = 0;
      if (++hk == (int)p.c.heads) {
        hk = 0;
        do r = load_req(p, ++b);
        while ((nt = tiles_of<R>(p, r)) == 0 && b < p.B - 1);
      }
    }
    s = tile_span<R, CH>(p, r, tile);
  }
};

// The line's [0, C) units over nc teams: team i has [C i / nc, C (i + 1) / nc); the team that
// has unit u.
__device__ __forceinline__ unsigned long long team_start(unsigned long long C, int nc, int i) { return C * i / nc; }
__device__ __forceinline__ int team_of(unsigned long long C, int nc, unsigned long long u) {
  return (int)(((u + 1) * nc - 1) / C);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The four bytes of w as float16 numbers, two to a word. Exact: int8 through 1024 + (byte + 128),
// whose float16 step is 1, the long published way to put a byte into a mantissa (the word
// already xor-ed by biased()); e4m3 is a subset of float16.
template <bool E4M3>
__device__ __forceinline__ void half4_of(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    const uint32_t u = __byte_perm(w, 0x64646464u, 0x4140), v = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 z = __half2half2(__ushort_as_half(0x6480));
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&u), z), y = __hsub2(*reinterpret_cast<const __half2*>(&v), z);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
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

// Four channels of a query row (row = query * G + head in the group).
template <bool BF16>
__device__ __forceinline__ void store_row(const AttnParams& p, const Req& r, int hk, int row, int ch, float4 a) {
  const int64_t at = ((int64_t)(r.q0 + row / p.G) * p.Hq + hk * p.G + row % p.G) * p.c.dh + ch;
  if constexpr (BF16) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(a.x, a.y), y = __floats2bfloat162_rn(a.z, a.w);
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  } else {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at) = make_float4(a.x, a.y, a.z, a.w);
  }
}

// The kernel for long rows of bf16 queries (kv8_prompt.cu): whether it takes a call with up to
// `rows` query rows a request and kv head and `all_rows` over all, the floats of one of its
// slots, and its launch.
bool prompt_takes(bool bf16, int64_t dh, int64_t rows, int64_t all_rows);
size_t prompt_slot_floats(int64_t dh);
wina_status_t launch_prompt(AttnParams& p, cudaStream_t s);

constexpr int kMaxCtas = 160;  // CTAs of either kernel, one per SM, at most

}  // namespace wina
