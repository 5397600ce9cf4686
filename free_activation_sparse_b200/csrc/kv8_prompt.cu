// Causal attention over the 8-bit paged cache for long rows of bf16 queries (prompt chunks):
// kv8_attention's tensor-core path on tcgen05 with accumulators in tensor memory.
//
//   S = Q K^T,  p = 2^(s c - m),  O += P V,  out = O / sum p      per block of 256 query rows
//
// Bound by the tensor cores and, about equally, by the exponentials (one per query row and
// key, 16 a clock and SM) once the bytes' conversion is shared by 256 rows.
#include <math.h>

#include <algorithm>
#include <atomic>

#include "kv8_attn.cuh"

namespace wina {

namespace {

constexpr int kRows = 256;        // query rows of a tile: two halves of 128
constexpr int kKeys = 128;        // keys of a chunk
constexpr int kThreads = 640;     // warps 0-3, 4-7: softmax of a half; 8-15: bytes; 16: matrix products
constexpr int kInfo = 4;          // chunks whose factors are kept
constexpr int kPartMin = 4;       // units of the line of work in a CTA's part, at least
// Registers a thread, of the 96 (640 threads) that it is launched with.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 136, kByteRegs = 80, kMmaRegs = 40;
static_assert(256 * kSoftmaxRegs + 256 * kByteRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs, "register split");
constexpr float kOffLog2 = 7.f;   // weights are held times 2^7 ...
constexpr float kLazyLog2 = 8.f;  // ... and may outgrow the reference maximum by 2^8 before O is rescaled
constexpr float kByteUp = 8.f;    // bytes are held times 8 scale / reference, the reference kept
constexpr float kGrow = 16.f;     // until a scale is 16 times as large

template <int DH>
struct PromptShape {
  static constexpr int TILE = kKeys * DH * 2;              // bytes of a chunk's keys (values) as float16
  static constexpr int QTILE = 128 * DH * 2;               // bytes of a half's queries
  static constexpr size_t SMEM = 1024 + 2 * QTILE + 4 * TILE;
  static constexpr uint32_t O_COL = 256;                   // tensor memory: S of both halves, then O of both
};

struct Info {
  float kfac;   // what a score is to be multiplied by besides its row's factor
  float sref;   // the value scales' reference
  uint32_t bad; // 16-key groups without a page
  uint32_t pad;
};

// Instruction descriptor of kind::f16 with float16 operands, float32 D, A K-major, B K-major
// or N-major, 128 x N.
constexpr uint32_t idesc_f16(int N, int b_n_major) {
  return (1u << 4) | ((uint32_t)b_n_major << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16, issued by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  const uint32_t z = 0u;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(z), "r"(z), "r"(z), "r"(z)
      : "memory");
}

// 32 lanes x 32 consecutive columns of tensor memory, to and from registers.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]),
        "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]),
        "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]),
      "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Byte offset of the 16-byte piece c (8 numbers) of row r in an operand tile of 128 rows: blocks
// of 64 numbers, 128 bytes a row, 128-byte swizzle.
__device__ __forceinline__ uint32_t operand_at(int r, int c) { return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4); }

// Four bytes as float16 numbers times f (two alike): exact where f is a power of two and the
// result no subnormal number.
template <bool E4M3>
__device__ __forceinline__ uint2 scaled_half4(uint32_t w, __half2 f) {
  uint32_t lo, hi;
  half4_of<E4M3>(biased<E4M3>(w), lo, hi);
  const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&lo), f), y = __hmul2(*reinterpret_cast<const __half2*>(&hi), f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
}

// Two float32 numbers at a time: a * b + c, a + b; the larger of three.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
// tanh x = 1 - 2 / (1 + e^(2 x)), off by at most 2^-22.
__device__ __forceinline__ float tanh_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(x * (2.f * kLog2e))));
  return fmaf(-2.f, r, 1.f);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

}  // namespace

// One CTA per SM on an equal part of the line of work (tiles of 256 query rows of one request
// and kv head, row = query * G + head of the group, times chunks of 128 keys), joined like the
// parts of k_kv8_attn_split. Two halves of 128 rows take turns: while one's softmax runs, the
// tensor cores work for the other.
//   warps 8-15 (bytes): a chunk's keys and values from the pages into shared memory as float16
//     times 8 scale / reference, the reference being the first chunk's largest scale, raised
//     when a scale passes 16 times it, so a score needs one factor per row and chunk and a weight
//     none. Exact for power-of-two scales down to 2^-27 (int8; e4m3, whose numbers start at 2^-9:
//     2^-18) of the reference: 8 * 2^-27 is float16's least number. Loads run a chunk ahead.
//   warp 16: S = Q K^T of either half as soon as its last P has been used, O += P V as soon as P
//     is there (P is the A operand from tensor memory, in the place of S).
//   warps 0-3, 4-7 (softmax, a thread per row): the row's maximum in one pass over S, the
//     weights as float16 in a second; O is rescaled only when a maximum outgrows its
//     reference by 2^8, a published idea (a weight keeps 11 bits from 2^15 down to 2^-14).
// Queries are float16 times a power of two per row (exact for bf16 within 2^28 of the row's
// largest). Places without a page or outside the tile's keys are zeros. A half whose bytes of a
// page are no numbers (kv8_write stores none) may get NaN where it does not see them.
//
// 4 chunks of up to 2048 queries behind 2 K to 6 K keys (32 / 8 heads of 128, 0.52 TFLOP): 0.80 ms,
// 650 TFLOP/s; a step of 128 keys takes 5.4 K cycles, of which the tensor cores work 2.1 K. What
// holds it is the chain of a half: products 1.6 K cycles with their hand-overs, maxima 0.9 K,
// weights 2.5 K; with the conversions, the exponentials and the first pass left out together it
// still takes 0.70 ms. Slower: four softmax warps a quarter (1.02 ms, spills), S by 64 keys in
// two places a half (1.00 ms, twice the hand-overs), both passes unrolled (1.23 ms, instruction
// caches; with four warps for the bytes and no packed arithmetic besides, 1.74 ms: four such
// warps were not tried with the short loops).
template <bool E4M3, int DH>
__global__ void __launch_bounds__(kThreads, 1) k_kv8_attn_prompt(const AttnParams p) {
  using Sh = PromptShape<DH>;
  constexpr int TILE = Sh::TILE, QTILE = Sh::QTILE;
  extern __shared__ unsigned char smraw[];
  __shared__ uint32_t red[32];
  __shared__ uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], info_full[kInfo], s_full[2], p_full[2], q_full[2], o_full[2];
  __shared__ Info s_info[kInfo];
  __shared__ uint32_t s_taddr, s_last;
  __shared__ int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t sbase = (tc::smem_u32(smraw) + 1023u) & ~1023u;
  unsigned char* sm = smraw + (sbase - tc::smem_u32(smraw));
  unsigned char* const qs = sm;                      // two halves' queries
  unsigned char* const ks = sm + 2 * QTILE;          // two chunks' keys
  unsigned char* const vs = ks + 2 * TILE;           // two chunks' values
  uint32_t* pre = reinterpret_cast<uint32_t*>(vs + 2 * TILE);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&k_full[i], 256u);
      tc::mbar_init(&v_full[i], 256u);
      tc::mbar_init(&k_empty[i], 1u);
      tc::mbar_init(&v_empty[i], 1u);
      tc::mbar_init(&s_full[i], 1u);
      tc::mbar_init(&p_full[i], 128u);
      tc::mbar_init(&q_full[i], 128u);
      tc::mbar_init(&o_full[i], 1u);
    }
    for (int i = 0; i < kInfo; ++i) tc::mbar_init(&info_full[i], 1u);
    tc::mbar_init_fence();
    s_abort = 0;
  }
  const bool fits = cost_prefix<kThreads, kRows, kKeys>(p, pre, red);
  const unsigned long long C = (unsigned long long)pre[pre_entries(p.B) - 1] * p.c.heads;
  if (fits) zero_rows<true>(p);
  if (!fits || C == 0) {
    if (!fits && blockIdx.x == 0 && tid == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
    return;
  }
  // a team's part is worth kPartMin units, so that few tiles are not cut into many parts to join
  const int nc = (int)min((unsigned long long)gridDim.x, max(1ull, C / kPartMin)), team = blockIdx.x;
  if (team >= nc) return;
  if (warp == 16) tc::tmem_alloc(&s_taddr, 512u);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t taddr = s_taddr;
  const unsigned long long u0 = team_start(C, nc, team), u1 = team_start(C, nc, team + 1);

  using W = Walk<kRows, kKeys>;
  auto part = [&](const W& w, int& from, int& to) { w.part(p, u0, u1, from, to); };
  // A wait that ran out (1 s) makes every later wait of the CTA return at once; all loops end by
  // their counts.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (*(volatile int*)&s_abort) return;
    if (!tc::mbar_wait(bar, parity)) {
      s_abort = 1;
      record_status(p.status, WINA_ERR_TIMEOUT);
    }
  };
  W w;

  if (warp >= 8 && warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kByteRegs));
    w.locate(p, pre, u0);
    // ---------------- bytes ----------------
    // warp 8 + d has 16-key group d of every chunk: one run of a page
    constexpr int PPR = DH / 16;         // 16-byte pieces of a row of bytes
    constexpr int RPI = 32 / PPR;        // rows of a warp's load
    constexpr int N = 16 / RPI;          // loads of 16 keys
    const int d = warp - 8, lr = lane / PPR, lc = lane % PPR;
    const int page_mask = (1 << p.shift) - 1;
    uint4 kr[N], vr[N];
    // loads of one side of this warp's group; head: its (page, head), -1 where there is none
    auto load = [&](int64_t head, int key0, int lo, int hi, const void* base, uint4 (&r)[N]) {
      const int key = key0 + 16 * d;
      const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(base) +
                                                        ((head << p.shift) + (key & page_mask)) * DH) + lane;
      const bool all = head >= 0 && key >= lo && key + 16 <= hi;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = key + i * RPI + lr;
        r[i] = make_uint4(0, 0, 0, 0);
        if (all || (head >= 0 && k >= lo && k < hi)) r[i] = __ldg(src + 32 * i);
      }
    };
    // One side into its tile, times f. The lanes of a row's second half store their pieces in the
    // other order, so that a row's eight lanes fall on different banks. (Places without a byte
    // were loaded as 0, which either format shows as 0.)
    const bool swap = lc & 4;
    const int c0 = 2 * lc + (swap ? 1 : 0), c1 = 2 * lc + (swap ? 0 : 1);
    const uint32_t at0 = operand_at(16 * d + lr, c0), at1 = operand_at(16 * d + lr, c1);
    auto store = [&](const uint4 (&r)[N], unsigned char* tile, float f) {
      const __half2 m = __float2half2_rn(f);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // row i * RPI further on: 128 bytes a row, and another permutation where RPI is 4
        const uint32_t flip = RPI == 4 && (i & 1) ? 64u : 0u;
        const uint2 a = scaled_half4<E4M3>(swap ? r[i].z : r[i].x, m), b = scaled_half4<E4M3>(swap ? r[i].w : r[i].y, m);
        *reinterpret_cast<uint4*>(tile + (at0 ^ flip) + i * RPI * 128) = make_uint4(a.x, a.y, b.x, b.y);
        const uint2 e = scaled_half4<E4M3>(swap ? r[i].x : r[i].z, m), g = scaled_half4<E4M3>(swap ? r[i].y : r[i].w, m);
        *reinterpret_cast<uint4*>(tile + (at1 ^ flip) + i * RPI * 128) = make_uint4(e.x, e.y, g.x, g.y);
      }
    };
    int c, to;
    part(w, c, to);
    // The chunk at or after c in the walk, with the page indices of its groups (lanes 0-7) on
    // their way.
    struct Next {
      bool any, used;
      int pg, hk, key0, lo, hi;
      unsigned long long at;
    };
    auto seek = [&]() {
      Next n;
      n.any = true;
      while (c >= to) {
        if (w.at + w.len(p) >= u1) {
          n.any = false;
          return n;
        }
        w.next(p);
        part(w, c, to);
      }
      n.key0 = c * kKeys;
      n.lo = w.s.lo;
      n.hi = w.s.hi;
      n.hk = w.hk;
      n.at = w.at;
      const int key = n.key0 + 16 * lane;
      n.used = lane < 8 && key < n.hi && key + 16 > n.lo;
      n.pg = n.used ? __ldg(p.table + (int64_t)w.b * p.width + (key >> p.shift)) : -1;
      ++c;
      return n;
    };
    auto head_of = [&](const Next& n) {  // of group `lane`
      return n.pg >= 0 && n.pg < p.c.n_pages ? (int64_t)n.pg * p.c.heads + n.hk : (int64_t)-1; };
    // chunk `it` is stored while chunk it + 1 is loaded and the pages of chunk it + 2 are found
    Next n = seek();
    bool any = n.any;
    unsigned long long at = n.at, tile_at = ~0ull;
    int64_t head = any ? head_of(n) : -1;
    uint32_t bad = __ballot_sync(0xffffffffu, any && n.used && head < 0);
    float kscale = 0.f, vscale = 0.f, kref = 0.f, sref = 0.f;
    if (any) {
      const int64_t mine = __shfl_sync(0xffffffffu, head, d);
      load(mine, n.key0, n.lo, n.hi, p.c.k, kr);
      load(mine, n.key0, n.lo, n.hi, p.c.v, vr);
      if (head >= 0) {
        kscale = __ldg(p.c.k_scale + head);
        vscale = __ldg(p.c.v_scale + head);
      }
      n = seek();
    }
    for (int it = 0; any; ++it) {
      const int st = it & 1;
      if (bad && lane == 0 && warp == 8) record_status(p.status, WINA_ERR_INVALID_ARG);
      if (tile_at != at) {  // a new tile: references start anew
        tile_at = at;
        kref = sref = 0.f;
      }
      // largest finite scales of the chunk
      float km = fabsf(kscale), vm = fabsf(vscale);
      const bool lost = !(vm < INFINITY);  // no finite value scale: the scores say so, the values are 0
      if (!(km < INFINITY)) km = 0.f;
      if (lost) vm = 0.f;
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) {
        km = fmaxf(km, __shfl_xor_sync(0xffffffffu, km, o));
        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, o));
      }
      km = __shfl_sync(0xffffffffu, km, 0);
      vm = __shfl_sync(0xffffffffu, vm, 0);
      if (km > kGrow * kref || kref == 0.f) kref = fmaxf(km, 1.17549435e-38f);
      if (vm > kGrow * sref || sref == 0.f) sref = fmaxf(vm, 1.17549435e-38f);
      float kf = lost ? __uint_as_float(0x7fc00000u) : kByteUp * (kscale / kref), vf = lost ? 0.f : kByteUp * (vscale / sref);
      kf = __shfl_sync(0xffffffffu, kf, d);
      vf = __shfl_sync(0xffffffffu, vf, d);
      // keys
      if (it >= 2) wait(&k_empty[st], (uint32_t)((it / 2 - 1) & 1));
      if (tid == 8 * 32) {
        s_info[it % kInfo] = Info{kref / kByteUp, sref / kByteUp, bad, 0u};
        tc::mbar_arrive(&info_full[it % kInfo]);
      }
      __syncwarp();
      store(kr, ks + st * TILE, kf);
      fence_async_smem();
      tc::mbar_arrive(&k_full[st]);
      any = n.any;
      int64_t mine = -1;
      if (any) {
        head = head_of(n);
        at = n.at;
        mine = __shfl_sync(0xffffffffu, head, d);
        load(mine, n.key0, n.lo, n.hi, p.c.k, kr);
      }
      // values
      if (it >= 2) wait(&v_empty[st], (uint32_t)((it / 2 - 1) & 1));
      store(vr, vs + st * TILE, vf);
      fence_async_smem();
      tc::mbar_arrive(&v_full[st]);
      if (any) {
        load(mine, n.key0, n.lo, n.hi, p.c.v, vr);
        kscale = head >= 0 ? __ldg(p.c.k_scale + head) : 0.f;
        vscale = head >= 0 ? __ldg(p.c.v_scale + head) : 0.f;
        bad = __ballot_sync(0xffffffffu, n.used && head < 0);
        n = seek();
      }
    }
  } else if (warp >= 16) {
    // ---------------- matrix products (one thread) ----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == 16 && lane == 0) {
      w.locate(p, pre, u0);
      const uint32_t id_qk = idesc_f16(kKeys, 0), id_pv = idesc_f16(DH, 1);
      int it = 0, tiles = 0, halves1 = 0, pn = 0, pn1 = 0;
      auto qk = [&](int h, int st) {
        const uint32_t q0 = tc::smem_u32(qs) + h * QTILE, k0 = tc::smem_u32(ks) + st * TILE;
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384u + (kk & 3) * 32u;
          tc::mma_bf16(taddr + h * 128u, tc::sw128_desc(q0 + off, 16u, 1024u), tc::sw128_desc(k0 + off, 16u, 1024u), id_qk, kk > 0);
        }
        tc::mma_commit(&s_full[h]);
      };
      auto pv = [&](int h, int st, bool first) {
        const uint32_t v0 = tc::smem_u32(vs) + st * TILE;
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_ts(taddr + Sh::O_COL + h * 128u, taddr + h * 128u + kk * 8u, tc::sw128_desc(v0 + kk * 2048u, 16384u, 1024u), id_pv,
                 !(first && kk == 0));
      };
      for (;;) {
        int from, to;
        part(w, from, to);
        if (from < to) {
          const int nh = w.r.nq * p.G - w.tile * kRows > 128 ? 2 : 1;
          for (int h = 0; h < nh; ++h) wait(&q_full[h], (uint32_t)((h ? halves1 : tiles) & 1));
          ++tiles;
          halves1 += nh - 1;
          wait(&k_full[it & 1], (uint32_t)((it / 2) & 1));
          tc::tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < nh; ++h) qk(h, it & 1);
          tc::mma_commit(&k_empty[it & 1]);
          for (int c = from; c < to; ++c, ++it) {
            const int st = it & 1, nst = (it + 1) & 1;
            wait(&v_full[st], (uint32_t)((it / 2) & 1));
            if (c + 1 < to) wait(&k_full[nst], (uint32_t)(((it + 1) / 2) & 1));
#pragma unroll 1
            for (int h = 0; h < nh; ++h) {
              wait(&p_full[h], (uint32_t)((h ? pn1++ : pn++) & 1));
              tc::tc_fence_after();
              pv(h, st, c == from);
              if (c + 1 < to) qk(h, nst);
              else tc::mma_commit(&o_full[h]);
            }
            tc::mma_commit(&v_empty[st]);
            if (c + 1 < to) tc::mma_commit(&k_empty[nst]);
          }
        }
        if (w.at + w.len(p) >= u1) break;
        w.next(p);
      }
      // nothing is in flight when the tensor memory is given back
      if (it > 0) tc::mbar_wait(&v_empty[(it - 1) & 1], (uint32_t)(((it - 1) / 2) & 1));
    }
  } else {
    // ---------------- softmax: half h, a thread per row ----------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    w.locate(p, pre, u0);
    const int h = warp >> 2, lrow = tid & 127;
    const uint32_t tm = taddr + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = tm + h * 128u, to_ = tm + Sh::O_COL + h * 128u;
    int it = 0, sn = 0, on = 0;
    for (;;) {
      int from, to;
      part(w, from, to);
      const int rows = min(kRows, w.r.nq * p.G - w.tile * kRows);
      if (from < to && rows > h * 128) {
        const int row = min(w.tile * kRows + h * 128 + lrow, w.tile * kRows + rows - 1);  // rows behind the last: copies
        const int i = row / p.G, pos0 = w.r.kv - w.r.n, lim = pos0 + i + 1, low = p.window > 0 ? lim - p.window : 0;
        // queries
        float fac;
        {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(p.q) + (int64_t)(w.r.q0 + i) * p.ld_q + (int64_t)(w.hk * p.G + row % p.G) * DH;
          uint4 r[DH / 8];
          uint32_t big = 0;
#pragma unroll
          for (int j = 0; j < DH / 8; ++j) {
            r[j] = __ldg(reinterpret_cast<const uint4*>(src) + j);
            const uint32_t u[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) big = max(big, max(u[e] & 0x7fffu, (u[e] >> 16) & 0x7fffu));
          }
          // the row's largest number goes to [2^14, 2^15)
          int ex = (int)(big >> 7);
          ex = ex == 255 ? 127 : max(15, ex);
          const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - ex) << 23);
          fac = __fdiv_rn(1.f, up) * p.scale * (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
          unsigned char* dst = qs + h * QTILE;
#pragma unroll
          for (int j = 0; j < DH / 8; ++j) {
            const uint32_t u[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = pack_half2(__uint_as_float(u[e] << 16) * up, __uint_as_float(u[e] & 0xffff0000u) * up);
            *reinterpret_cast<uint4*>(dst + operand_at(lrow, j)) = make_uint4(o[0], o[1], o[2], o[3]);
          }
          fence_async_smem();
          tc::tc_fence_before();
          tc::mbar_arrive(&q_full[h]);
        }
        // chunks between these need no masks
        const int first_lim = pos0 + (w.tile * kRows + h * 128) / p.G + 1;
        const int last_row = w.tile * kRows + min(rows, h * 128 + 128) - 1;
        const int last_low = max(w.s.lo, p.window > 0 ? pos0 + last_row / p.G + 1 - p.window : 0);
        float m = -INFINITY, l = 0.f, sref = 0.f;
        for (int c = from; c < to; ++c, ++it) {
          wait(&s_full[h], (uint32_t)(sn++ & 1));
          tc::tc_fence_after();
          // after S, so that the barrier is at this chunk's phase: a half that had no rows in the
          // tile before comes here many phases early, and could not tell them apart
          wait(&info_full[it % kInfo], (uint32_t)((it / kInfo) & 1));
          const Info info = s_info[it % kInfo];
          const int key0 = c * kKeys;
          const bool masked = info.bad || key0 < last_low || key0 + kKeys > first_lim;
          const float cf = fac * info.kfac;
          // Both passes are loops of 32 columns, kept short: the three roles' code together has to
          // stay in the instruction caches (with everything unrolled, warps waited for
          // instructions a third of the time).
          uint32_t v[32];
          float x0 = -INFINITY, x1 = -INFINITY;
          // places that the row does not see
          auto leave_out = [&](int col) {
            const int past = lim - (key0 + col), before = low - (key0 + col);
            const uint32_t off = info.bad >> (col >> 4);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (e >= past || e < before || ((off >> (e >> 4)) & 1)) v[e] = 0xff800000u;
          };
#pragma unroll 1
          for (int col = 0; col < kKeys; col += 32) {
            tmem_ld32(ts + col, v);
            tc::tmem_ld_wait();
            if (masked) leave_out(col);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              x0 = max3(x0, __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
              x1 = max3(x1, __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
            }
          }
          float x = fmaxf(x0, x1) * cf;
          if (p.softcap > 0.f) x = tanh_fast(x) * (p.softcap * kLog2e);
          const bool raise = x > m + kLazyLog2 || (m == -INFINITY && x > -INFINITY);
          const float mn = raise ? x : m;
          if (__any_sync(0xffffffffu, raise) || info.sref != sref) {
            const float al = raise ? ex2(m - mn) : 1.f;
            l *= al;
            if (c > from) {
              const float f = al * (sref / info.sref);
#pragma unroll 1
              for (int j = 0; j < DH; j += 32) {
                tmem_ld32(to_ + j, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                tmem_st32(to_ + j, v);
              }
              tmem_st_wait();
            }
            m = mn;
            sref = info.sref;
          }
          const float mb = m == -INFINITY ? 0.f : m - kOffLog2;
          float2 l0 = make_float2(0.f, 0.f), l1 = l0;
          // weights as float16 in the place of scores already read
#pragma unroll 1
          for (int col = 0; col < kKeys; col += 32) {
            tmem_ld32(ts + col, v);
            tc::tmem_ld_wait();
            if (p.softcap > 0.f) {
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(tanh_fast(__uint_as_float(v[e]) * cf) * (p.softcap * kLog2e) - mb);
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 y = fma2(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), make_float2(cf, cf), make_float2(-mb, -mb));
                v[e] = __float_as_uint(y.x);
                v[e + 1] = __float_as_uint(y.y);
              }
            }
            if (masked) leave_out(col);
            uint32_t o[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 y = make_float2(ex2(__uint_as_float(v[e])), ex2(__uint_as_float(v[e + 1])));
              if (e & 2) l1 = add2(l1, y);
              else l0 = add2(l0, y);
              o[e / 2] = pack_half2(y.x, y.y);
            }
            tmem_st16(ts + col / 2, o);
          }
          l += (l0.x + l0.y) + (l1.x + l1.y);
          tmem_st_wait();
          tc::tc_fence_before();
          tc::mbar_arrive(&p_full[h]);
        }
        // the tile's (or this part's) sums
        wait(&o_full[h], (uint32_t)(on++ & 1));
        tc::tc_fence_after();
        const bool whole = from == w.s.c0 && to == w.s.c1, mine = h * 128 + lrow < rows;
        float* slot = p.slots + (size_t)(2 * team + (from == w.s.c0 ? 1 : 0)) * p.slot_floats;
        // over the row's weights so far, whole or part: plain sums would pass float32's range long before
        // their quotient does (and in two factors, whose product can be too small for float32)
        const float f = l == 0.f ? 0.f : 1.f / l;
        const int64_t at = ((int64_t)(w.r.q0 + i) * p.Hq + w.hk * p.G + row % p.G) * DH;
        uint32_t o[32];
#pragma unroll 1
        for (int j = 0; j < DH; j += 32) {
          tmem_ld32(to_ + j, o);
          tc::tmem_ld_wait();
          if (!mine) continue;
          if (whole) {
            uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at + j);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[8 * q + 2 * e]) * f * sref, __uint_as_float(o[8 * q + 2 * e + 1]) * f * sref);
                x[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              d[q] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          } else {
            float4* d = reinterpret_cast<float4*>(slot + (size_t)(h * 128 + lrow) * DH + j);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              d[q] = make_float4(__uint_as_float(o[4 * q]) * f * sref, __uint_as_float(o[4 * q + 1]) * f * sref,
                                 __uint_as_float(o[4 * q + 2]) * f * sref, __uint_as_float(o[4 * q + 3]) * f * sref);
          }
        }
        if (!whole && mine) {
          slot[kRows * DH + h * 128 + lrow] = m;
          slot[kRows * DH + kRows + h * 128 + lrow] = l;
        }
        tc::tc_fence_before();  // O has been read before the next tile's first product, which waits for P
      } else {
        it += max(0, to - from);  // the other half's chunks
        if (w.empty_of(u0, u1))
          for (int j = tid; j < rows * DH / 4; j += 256)
            store_row<true>(p, w.r, w.hk, w.tile * kRows + j / (DH / 4), (j % (DH / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
      }
      if (from < to && !(from == w.s.c0 && to == w.s.c1)) {
        // both halves together: the last of the tile's teams joins the parts in order
        const int ta = team_of(C, nc, w.at + p.tile_cost), tb = team_of(C, nc, w.at + w.len(p) - 1), parts = tb - ta + 1;
        __threadfence();
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 0) {
          s_last = atomicAdd(p.counters + ta, 1u) == (unsigned)(parts - 1);
          if (s_last) p.counters[ta] = 0;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (s_last) {
          __threadfence();
          auto part_of = [&](int k) { return p.slots + (size_t)(2 * (ta + k) + (k == 0 ? 1 : 0)) * p.slot_floats; };
          // a thread per row: each part's factor, in the place of its maximum
          if (tid < rows) {
            float M = -INFINITY, L = 0.f;
#pragma unroll 4
            for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(part_of(k) + kRows * DH + tid));
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
              const float mk = __ldcg(part_of(k) + kRows * DH + tid), lk = __ldcg(part_of(k) + kRows * DH + kRows + tid);
              L += lk == 0.f ? 0.f : lk * ex2(mk - M);
            }
            const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll 4
            for (int k = 0; k < parts; ++k) {
              const float mk = __ldcg(part_of(k) + kRows * DH + tid), lk = __ldcg(part_of(k) + kRows * DH + kRows + tid);
              __stcg(part_of(k) + kRows * DH + tid, lk == 0.f ? 0.f : lk * ex2(mk - M) * inv);
            }
          }
          asm volatile("bar.sync 1, 256;" ::: "memory");
          // eight pieces of a thread at a time, so that their loads do not wait for one another
          // (one at a time, a tile of four parts took 50 us)
          constexpr int U = 8;
          for (int j0 = tid; j0 < rows * DH / 4; j0 += 256 * U) {
            float4 a[U];
#pragma unroll
            for (int u = 0; u < U; ++u) a[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = 0; k < parts; ++k) {
              const float* q = part_of(k);
              float4 x[U];
              float f[U];
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const int j = j0 + 256 * u;
                f[u] = 0.f;
                if (j < rows * DH / 4) {
                  x[u] = __ldcg(reinterpret_cast<const float4*>(q) + j);
                  f[u] = __ldcg(q + kRows * DH + j / (DH / 4));
                }
              }
#pragma unroll
              for (int u = 0; u < U; ++u)
                if (j0 + 256 * u < rows * DH / 4) {
                  a[u].x += x[u].x * f[u];
                  a[u].y += x[u].y * f[u];
                  a[u].z += x[u].z * f[u];
                  a[u].w += x[u].w * f[u];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int j = j0 + 256 * u;
              if (j < rows * DH / 4) store_row<true>(p, w.r, w.hk, w.tile * kRows + j / (DH / 4), (j % (DH / 4)) * 4, a[u]);
            }
          }
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
      }
      if (w.at + w.len(p) >= u1) break;
      w.next(p);
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc::tc_fence_after();
    tc::tmem_dealloc(taddr, 512u);
  }
}

// More than 96 query rows a request and kv head, and 20 tiles at least over all: below that
// k_kv8_attn_split is as fast or faster (32 / 8 heads, 6 K keys: 4 requests of 24 queries 67 us
// against 70 here, of 128 queries 250 against 130; one request of 64 queries, 8 tiles, 51 against
// 82; 32 requests of 32 queries 242 against 172).
bool prompt_takes(bool bf16, int64_t dh, int64_t rows, int64_t all_rows) {
  return bf16 && dh <= 128 && rows > 96 && all_rows >= 20 * kRows;
}


size_t prompt_slot_floats(int64_t dh) { return (size_t)kRows * (dh + 2); }

wina_status_t launch_prompt(AttnParams& p, cudaStream_t s) {
  const int sms = device_sm_count();
  if (sms < 1) return WINA_ERR_CUDA;
  p.slot_floats = (int)prompt_slot_floats(p.c.dh);
  p.tiles = 0;
  p.tile_cost = 2;
  const bool e4 = p.c.format == KV8_E4M3;
  void (*kern)(const AttnParams) = p.c.dh == 64 ? (e4 ? k_kv8_attn_prompt<true, 64> : k_kv8_attn_prompt<false, 64>)
                                                : (e4 ? k_kv8_attn_prompt<true, 128> : k_kv8_attn_prompt<false, 128>);
  // the register split draws on what the kernel is launched with: never launch it with less
  static std::atomic<bool> checked[4];
  std::atomic<bool>& seen = checked[(p.c.dh == 64 ? 2 : 0) + (e4 ? 1 : 0)];
  if (!seen.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    const cudaError_t e = cudaFuncGetAttributes(&a, (const void*)kern);
    if (e != cudaSuccess) return cuda_status(e);
    if (a.numRegs < kLaunchRegs) return WINA_ERR_CUDA;
    seen.store(true, std::memory_order_relaxed);
  }
  const size_t smem = (p.c.dh == 64 ? PromptShape<64>::SMEM : PromptShape<128>::SMEM) + round_up((size_t)pre_entries(p.B) * 4, 16);
  return cuda_status(launch_kernel(kern, dim3((unsigned)std::min(sms, kMaxCtas)), dim3(kThreads), smem, s, false, p));
}

}  // namespace wina
