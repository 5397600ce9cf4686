// Causal attention over the 8-bit paged key/value cache (kv8_attention).
//
//   s_j = (q . k8_j) ks[page_j] scale;  out = sum_j p_j vs[page_j] v8_j / sum_j p_j,
//   p_j = exp(s_j - max)
//
// Two kernels. k_kv8_attn_split (here): single tokens, short spans, rows 256 wide, and float32
// prompts; bound by HBM: every key and value byte is read once per block of 8 or 16 query rows
// (the rows of a kv head's query group, so grouped queries share the read).
// k_kv8_attn_prompt (kv8_prompt.cu): prompt chunks of bf16 queries, on the tensor cores.
#include <math.h>

#include <algorithm>
#include <cmath>

#include "kv8_attn.cuh"

namespace wina {

// 16 bytes to shared memory, of which `bytes` are read and the rest zero, under an L2 policy.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes, uint64_t pol) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes), "l"(pol)
               : "memory");
}

// Four bytes to shared memory (zeros where `bytes` is 0).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// ------------------------------------------------------------------------------------
// k_kv8_attn_split
// ------------------------------------------------------------------------------------

constexpr int kMaxWarps = 12;               // consumer warps of a CTA, at most
constexpr int kMaxTeams = kMaxCtas * kMaxWarps;
constexpr int kMaxStages = 4;
constexpr float kPScaleLog2 = 14.f;         // weights are held times 2^14 (float16's middle)

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

// Byte offset of 16-byte piece c of row r in a staged group of 16 rows of DH bytes. The pieces
// are permuted so that both the key reads (8 lanes: 2 rows, 4 pieces) and the value reads (8
// lanes: 4 rows, 2 pieces) fall on different banks.
template <int DH>
__device__ __forceinline__ uint32_t staged(int r, int c) {
  if constexpr (DH == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else return (c >> 3) * 2048 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// The variants' sizes. The registers set the number of warps (a tile's sums and
// queries: 16 rows, or rows of 256, or queries in two parts take the most); the shared memory
// the depth of their rings.
template <bool BF16, int DH, int NT>
struct SplitShape {
  static constexpr int CH = DH == 256 ? 16 : 32;          // keys of a chunk
  static constexpr int R = 8 * NT;                        // query rows of a tile
  static constexpr int STAGE = 2 * CH * DH;               // bytes of a chunk, keys and values
  static constexpr int NCW = NT * DH == 256 ? 8 : 12;     // warps, of 255 or 168 registers a thread
  static constexpr int THREADS = 32 * NCW;
  static constexpr int S = DH == 64 ? 4 : NCW == 8 ? 3 : 2;  // chunks of a warp's ring
  static constexpr int RPR = DH == 256 ? 2 : 4;           // rows joined at a time
  static constexpr int MERGE = NCW * RPR * DH * 4;        // bytes of the merge buffer
  static constexpr size_t SMEM = (size_t)NCW * S * STAGE + MERGE;
};

// One CTA per SM. The work (tiles of 8 NT query rows of one request and kv head, times the
// chunks of CH keys they see) is a line cut into equal parts, one for each team, so that one long
// sequence fills the GPU and a ragged batch is balanced. A team is a whole CTA, whose warps take
// a tile's chunks in turn (few tiles), or one warp (many tiles, whose fixed costs then run side by
// side). Each warp copies its own chunks into its own ring (cp.async, 16 bytes a lane; places
// outside the tile's keys become zeros and are not read), running ahead across tiles, so that
// loads stay in flight while tiles are joined. (A warp that feeds the others by tensor copies was
// slower: a copy of 16 x 128 bytes takes it 80 to 116 cycles.)
//
// Per chunk, with keys as the rows of the matrix instruction, so that 8 query rows cost half
// of what 16 do:
//   S^T = K Q^T   bytes to float16 (exact), queries as float16 times a power of two per row
//                 (bf16: exact; float32: two float16 parts, 2^-22 of the row's largest), the
//                 channels in the order the 16-byte reads deliver them, which the sum does
//                 not mind;
//   running max, p = 2^(s - max + 14), sum p in float32;
//   O^T += V^T P^T with P = p vs / sref in float16 (float32: two parts), sref the largest
//                 value scale met so far: P keeps 11 bits down to 2^-28 of the row's largest weight
//                 (22 down to 2^-16) and is within 2^-39 of it below; O is rescaled where max or
//                 sref grow.
// The matrix instruction's additions to its accumulator do not round to nearest, so for float32
// queries a chunk's sums are made apart and added in float32, and the second parts' scores apart
// from the first's (2-norm errors at 9 K keys: 0.4e-6 to 0.9e-6, and 0.7e-6 to 3.2e-6 without, for
// 2 % of the time, or 15 % with 16 rows).
// The bytes' conversion and the softmax, some 420 instructions a chunk of 32 keys in one
// dependent stream, are what a warp spends its time on; twelve warps hide its latency (64 long
// contexts, 1.3 GB: 208 us, 6.3 TB/s; 264 us with eight warps).
// A team's warps' (max, sum, O / sum) are joined in shared memory in warp order (their sums tell
// which warps have keys; a warp of NaN scores has no maximum but a sum); a tile cut by a
// part's end is left in the workspace, and the last team of that tile to arrive joins the
// parts in order. No team waits for another.
template <bool BF16, bool E4M3, int DH, int NT, bool WARPS>
__global__ void __launch_bounds__(SplitShape<BF16, DH, NT>::THREADS, 1)
    k_kv8_attn_split(const AttnParams p) {
  using Sh = SplitShape<BF16, DH, NT>;
  constexpr int CH = Sh::CH, R = Sh::R, STAGE = Sh::STAGE, NCW = Sh::NCW, S = Sh::S, RPR = Sh::RPR;
  constexpr int TEAM = WARPS ? 1 : NCW;       // warps of a team
  constexpr int MT = CH / 16;                 // 16-key groups of a chunk
  constexpr int KS = DH / 16;                 // k-steps of a score, and 16-channel tiles of O
  constexpr int KC = DH / 64;                 // 16-byte pieces of a key row per lane
  constexpr int PARTS = BF16 ? 1 : 2;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint32_t red[32];
  __shared__ float s_m[NCW][R], s_l[NCW][R];
  __shared__ float s_meta[NCW][S][4];         // ks, vs of a chunk's 16-key groups
  __shared__ uint32_t s_bad[NCW][S];
  __shared__ uint32_t s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  float* mbuf = reinterpret_cast<float*>(sm + (size_t)NCW * S * STAGE);
  uint32_t* pre = reinterpret_cast<uint32_t*>(sm + (size_t)NCW * S * STAGE + Sh::MERGE);
  if (!cost_prefix<Sh::THREADS, R, CH>(p, pre, red)) {
    if (blockIdx.x == 0 && tid == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
    return;
  }
  const unsigned long long C = (unsigned long long)pre[pre_entries(p.B) - 1] * p.c.heads;
  zero_rows<BF16>(p);
  if (C == 0) return;
  // The number of teams. A CTA that gets parts of two tiles pays a tile's fixed cost twice, so
  // with fewer tiles than CTAs it is a multiple of the tiles (each of equal tiles is then cut
  // alike, and no CTA has parts of two) unless that leaves too many idle; a part is worth at
  // least a chunk for each of the CTA's warps. (One sequence of 4096 tokens, 32 heads: 18.6 us
  // on all SMs, 16.7 on 128 of them.)
  const int teams = gridDim.x * (NCW / TEAM);
  int nc = teams;
  if (!WARPS && p.tiles <= teams) {
    const int k = (int)max(1ull, min((unsigned long long)(teams / p.tiles), (C / p.tiles + TEAM / 2) / TEAM));
    const int even = p.tiles * k;
    nc = (int)min((unsigned long long)teams, max((unsigned long long)p.tiles, C / TEAM));
    if (C / even <= C / nc + 20) nc = even;
  }
  nc = (int)min((unsigned long long)nc, C);  // every team has a unit, so that a tile's parts can be counted
  const int team = WARPS ? warp * gridDim.x + blockIdx.x : blockIdx.x, member = WARPS ? 0 : warp;
  if (team >= nc) return;
  const unsigned long long u0 = team_start(C, nc, team), u1 = team_start(C, nc, team + 1);

  using W = Walk<R, CH>;
  // of a team's chunks [from, to) this warp's are from + member, + TEAM, ...
  auto part = [&](const W& w, int& from, int& to) { w.part(p, u0, u1, from, to); };
  W w;  // the tile being computed
  w.locate(p, pre, u0);

  // ---- loading: the warp's next chunk, tile after tile ----
  // (the walk lies in shared memory: it is looked at when a tile ends, and would cost registers)
  __shared__ W s_walk[NCW];
  const uint64_t pol = l2_evict_first_policy();
  const int page_mask = (1 << p.shift) - 1;
  int pc, pto, plo, phi, phk;       // its chunk, and its tile's end, keys and head
  int pg0 = -1, pg1 = -1, pg_from;  // page indices of its tile's next chunks, one chunk to a lane
  bool more = true;
  auto load_pages = [&](const W& v) {
    pg_from = pc;
    const int64_t key = (int64_t)(pc + lane * TEAM) * CH;
    const int32_t* row = p.table + (int64_t)v.b * p.width;
    pg0 = key < v.s.hi && key + 16 > v.s.lo ? __ldg(row + (key >> p.shift)) : -1;
    if (MT == 2) pg1 = key + 16 < v.s.hi && key + 32 > v.s.lo ? __ldg(row + ((key + 16) >> p.shift)) : -1;
  };
  auto enter = [&](const W& v) {
    part(v, pc, pto);
    pc += member;
    plo = v.s.lo;
    phi = v.s.hi;
    phk = v.hk;
    load_pages(v);
    // the tile's queries, towards L2
    constexpr int LINES = DH * (BF16 ? 2 : 4) / 128;
    for (int i = member * 32 + lane; i < R * LINES; i += TEAM * 32) {
      const int rr = v.tile * R + i / LINES;
      if (rr < v.r.nq * p.G) {
        const int64_t at = (int64_t)(v.r.q0 + rr / p.G) * p.ld_q + (int64_t)(v.hk * p.G + rr % p.G) * DH;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(p.q) + at * (BF16 ? 2 : 4) + (i % LINES) * 128));
      }
    }
  };
  enter(w);
  if (lane == 0) s_walk[warp] = w;
  __syncwarp();
  // offsets of this lane's pieces: of its first copy, its key rows and its value rows
  constexpr int RB = DH == 64 ? 64 : 128;  // bytes from row to row of a staged block
  const uint32_t in_group = staged<DH>(lane / (DH / 16), lane % (DH / 16));
  const uint32_t k_at = staged<DH>(g, DH == 64 ? t : 2 * t), v_at = staged<DH>(2 * t, DH == 64 ? g >> 1 : g);
  // one chunk into `slot`
  auto issue = [&](int slot) {
    while (more && pc >= pto) {  // the next tile with a chunk for this warp
      W v = s_walk[warp];
      __syncwarp();
      if (v.at + v.len(p) >= u1) {
        more = false;
        break;
      }
      v.next(p);
      enter(v);
      if (lane == 0) s_walk[warp] = v;
      __syncwarp();
    }
    if (more) {
      if (pc - pg_from == 32 * TEAM) load_pages(s_walk[warp]);
      const int src = (pc - pg_from) / TEAM, key0 = pc * CH;
      uint32_t bad = 0;
      int64_t head[MT];  // (page, head) of each 16-key group, -1 where none is read
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const int pg = __shfl_sync(0xffffffffu, u ? pg1 : pg0, src);
        const bool used = key0 + 16 * u < phi && key0 + 16 * u + 16 > plo, ok = used && pg >= 0 && pg < p.c.n_pages;
        head[u] = ok ? (int64_t)pg * p.c.heads + phk : -1;
        if (used && !ok) bad |= 1u << u;
      }
      if (bad && lane == 0) record_status(p.status, WINA_ERR_INVALID_ARG);
      const uint32_t dst = tc::smem_u32(sm + (size_t)(warp * S + slot) * STAGE);
      constexpr int PPR = DH / 16, RPI = 32 / PPR, N = 16 / RPI;  // pieces of a row, rows and passes of a warp
      bool inside = key0 >= plo && key0 + CH <= phi;
#pragma unroll
      for (int u = 0; u < MT; ++u) inside = inside && head[u] >= 0;
      if (inside) {
        // a group is one run of a page: fixed offsets from one address
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          const int64_t from = ((head[u] << p.shift) + ((key0 + 16 * u) & page_mask)) * DH + lane * 16;
          const uint8_t *sk = reinterpret_cast<const uint8_t*>(p.c.k) + from, *sv = reinterpret_cast<const uint8_t*>(p.c.v) + from;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint32_t d = dst + u * 16 * DH + (in_group ^ (DH == 64 ? 0 : ((i * RPI) & 7) << 4)) + i * RPI * RB;
            cp_async16(d, sk + 512 * i, 16, pol);
            cp_async16(d + CH * DH, sv + 512 * i, 16, pol);
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll 1
          for (int i = 0; i < N; ++i) {
            const int row = i * RPI + lane / PPR, key = key0 + 16 * u + row;
            const bool on = head[u] >= 0 && key >= plo && key < phi;
            const int64_t from = on ? ((head[u] << p.shift) + (key & page_mask)) * DH + (lane % PPR) * 16 : 0;
            const uint32_t d = dst + u * 16 * DH + staged<DH>(row, lane % PPR);
            cp_async16(d, reinterpret_cast<const uint8_t*>(p.c.k) + from, on ? 16 : 0, pol);
            cp_async16(d + CH * DH, reinterpret_cast<const uint8_t*>(p.c.v) + from, on ? 16 : 0, pol);
          }
      }
      if (lane < 2 * MT) {
        const int64_t h = (MT == 2 && (lane & 1)) ? head[MT - 1] : head[0];
        cp_async4(tc::smem_u32(&s_meta[warp][slot][lane]), (lane >= MT ? p.c.v_scale : p.c.k_scale) + (h >= 0 ? h : 0), h >= 0 ? 4 : 0);
      }
      if (lane == 0) s_bad[warp][slot] = bad;
      pc += TEAM;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i);

  int it = 0;
  for (;;) {  // tiles
    int from, to;
    part(w, from, to);
    const int rows = min(R, w.r.nq * p.G - w.tile * R);
    if (from >= to) {
      if (w.empty_of(u0, u1))
        for (int i = member * 32 + lane; i < rows * DH / 4; i += 32 * TEAM)
          store_row<BF16>(p, w.r, w.hk, w.tile * R + i / (DH / 4), (i % (DH / 4)) * 4, make_float4(0.f, 0.f, 0.f, 0.f));
      if (w.at + w.len(p) >= u1) break;
      w.next(p);
      continue;
    }
    // queries: lane (g, t) has row g's pieces of channels as the keys' lanes t have them
    uint32_t qf[PARTS][NT][KS][2];
    float cr[NT][2];  // factor of a score, rows 2t and 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = nt * 8 + g, rr = w.tile * R + row;
      const int64_t at = (int64_t)(w.r.q0 + rr / p.G) * p.ld_q + (int64_t)(w.hk * p.G + rr % p.G) * DH;
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
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = f[j][4 * k + 2 * e] * up, y = f[j][4 * k + 2 * e + 1] * up;
            const __half2 h = __floats2half2_rn(x, y);
            qf[0][nt][j * 4 + k][e] = *reinterpret_cast<const uint32_t*>(&h);
            if constexpr (!BF16) {
              const float2 back = __half22float2(h);
              qf[PARTS - 1][nt][j * 4 + k][e] = pack_half2(x - back.x, y - back.y);
            }
          }
      const float fac = dn * p.scale * (p.softcap > 0.f ? 1.f / p.softcap : kLog2e);
      cr[nt][0] = __shfl_sync(0xffffffffu, fac, 8 * t);
      cr[nt][1] = __shfl_sync(0xffffffffu, fac, 8 * t + 4);
    }
    // chunks between these need no masks
    const int pos0 = w.r.kv - w.r.n;
    const int first_lim = pos0 + w.tile * R / p.G + 1;
    const int last_low = max(w.s.lo, p.window > 0 ? pos0 + (w.tile * R + rows - 1) / p.G + 1 - p.window : 0);

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

    for (int c = from + member; c < to; c += TEAM, ++it) {
      const int slot = it % S;
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
      __syncwarp();  // everybody's pieces are there, and the slot before this one is read
      issue((it + S - 1) % S);
      const unsigned char* kst = sm + (size_t)(warp * S + slot) * STAGE;
      const unsigned char* vst = kst + CH * DH;
      float s[NT][MT][4], s_low[NT][MT][4];  // (float32 queries' second parts apart: see below)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[nt][u][e] = s_low[nt][u][e] = 0.f;
#pragma unroll
      for (int u = 0; u < MT; ++u)
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          // piece 2 t + (j & 1) of block j / 2 (DH 64: piece t); row g + 8 is permuted like row g
          const unsigned char* at = kst + u * 16 * DH + (j >> 1) * 2048 + (k_at ^ ((j & 1) << 4));
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          const uint4 y = *reinterpret_cast<const uint4*>(at + 8 * RB);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a = biased<E4M3>(xs[k]), b = biased<E4M3>(ys[k]);
            uint32_t fr[4];
            half4_of<E4M3>(a, fr[0], fr[2]);
            half4_of<E4M3>(b, fr[1], fr[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int q = 0; q < PARTS; ++q)
                mma16816(q ? s_low[nt][u] : s[nt][u], fr, qf[q][nt][j * 4 + k][0], qf[q][nt][j * 4 + k][1]);
          }
        }
      float ks[MT], vs[MT];
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        ks[u] = s_meta[warp][slot][u];
        vs[u] = s_meta[warp][slot][MT + u];
        // values that no scale holds: the scores say so, since a weight may be too small to
        if (!(fabsf(vs[u]) < INFINITY)) ks[u] = __uint_as_float(0x7fc00000u);
      }
      const uint32_t bad = s_bad[warp][slot];
      const int key0 = c * CH;
      const bool masked = bad || key0 < last_low || key0 + CH > first_lim;
      // scores in units of log 2
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = (BF16 ? s[nt][u][e] : s[nt][u][e] + s_low[nt][u][e]) * (cr[nt][e & 1] * ks[u]);
            if (p.softcap > 0.f) x = tanhf(x) * (p.softcap * kLog2e);
            s[nt][u][e] = x;
          }
      if (masked) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the keys that row 2t + e sees
            const int lim = pos0 + (w.tile * R + min(nt * 8 + 2 * t + e, rows - 1)) / p.G + 1;
            const int low = p.window > 0 ? lim - p.window : 0;
#pragma unroll
            for (int u = 0; u < MT; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int key = key0 + 16 * u + g + h * 8;
                if (key >= lim || key < low || ((bad >> u) & 1)) s[nt][u][2 * h + e] = -INFINITY;
              }
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
        if (a < INFINITY) vmax = fmaxf(vmax, a);
      }
      if (__any_sync(0xffffffffu, grew) || vmax > sref) {
        inv_sref = __fdiv_rn(1.f, vmax);
        const float down = sref * inv_sref;
        sref = vmax;
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
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = ex2(s[nt][u][e] - mb[nt][e & 1]);
            l[nt][e & 1] += x[e];
            // a weight of 0 stays 0 under any scale
            x[e] = x[e] == 0.f ? 0.f : x[e] * ratio;
          }
          const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
          pf[0][nt][u][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&a));
          pf[0][nt][u][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&b));
          if constexpr (!BF16) {
            const float2 fa = __half22float2(a), fb = __half22float2(b);
            pf[PARTS - 1][nt][u][0] = transpose8x8(pack_half2(x[0] - fa.x, x[1] - fa.y));
            pf[PARTS - 1][nt][u][1] = transpose8x8(pack_half2(x[2] - fb.x, x[3] - fb.y));
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
            // row 2 t + (k & 1) + 8 (k >> 1)
            const unsigned char* at = vst + u * 16 * DH + h * 2048 + (v_at ^ (DH == 64 ? 0 : (k & 1) << 4)) + ((k & 1) + (k >> 1) * 8) * RB;
            if constexpr (DH == 64) {
              const uint2 v = *reinterpret_cast<const uint2*>(at + (g & 1) * 8);
              x[k][0] = v.x;
              x[k][1] = v.y;
            } else {
              const uint4 v = *reinterpret_cast<const uint4*>(at);
              x[k][0] = v.x;
              x[k][1] = v.y;
              x[k][2] = v.z;
              x[k][3] = v.w;
            }
#pragma unroll
            for (int q = 0; q < VW; ++q) x[k][q] = biased<E4M3>(x[k][q]);
          }
#pragma unroll
          for (int q = 0; q < VW; ++q) {
            // channels 4q, 4q + 1 of two keys side by side, then 4q + 2, 4q + 3
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a = __byte_perm(x[0][q], x[1][q], e ? 0x7362 : 0x5140);
              const uint32_t b = __byte_perm(x[2][q], x[3][q], e ? 0x7362 : 0x5140);
              uint32_t fr[4];
              half4_of<E4M3>(a, fr[0], fr[1]);
              half4_of<E4M3>(b, fr[2], fr[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if constexpr (BF16) {
                  mma16816(o[nt][h * 8 + 2 * q + e], fr, pf[0][nt][u][0], pf[0][nt][u][1]);
                } else {
                  float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                  for (int i = PARTS - 1; i >= 0; --i) mma16816(add, fr, pf[i][nt][u][0], pf[i][nt][u][1]);
#pragma unroll
                  for (int i = 0; i < 4; ++i) o[nt][h * 8 + 2 * q + e][i] += add[i];
                }
              }
            }
          }
        }
    }

    // ---- join the warps' parts of this tile ----
    const bool whole = from == w.s.c0 && to == w.s.c1;
    // this team's slot: a part that begins its tile elsewhere comes first
    float* slot = p.slots + (size_t)(2 * team + (from == w.s.c0 ? 1 : 0)) * p.slot_floats;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        l[nt][e] = x;
        if (!WARPS && g == 0) {
          s_m[warp][nt * 8 + 2 * t + e] = m[nt][e];
          s_l[warp][nt * 8 + 2 * t + e] = x;
        }
      }
    // Four channels of row (nt, e) over the row's weights so far. Parts are kept and joined so, not
    // as plain sums, which pass float32's range long before their quotient does.
    auto mean = [&](int nt, int j, int e) {
      const float inv = l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e];
      return make_float4(o[nt][j][e] * inv * sref, o[nt][j][e + 2] * inv * sref, o[nt][j + 1][e] * inv * sref,
                         o[nt][j + 1][e + 2] * inv * sref);
    };
    constexpr int CPL = DH == 64 ? 8 : 16;  // consecutive channels a lane has (of each 128)
    if constexpr (WARPS) {
      // lane (g, t): rows 2t, 2t + 1, channels g * CPL ..
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = nt * 8 + 2 * t + e;
          if (row >= rows) continue;
#pragma unroll
          for (int h = 0; h < (DH == 256 ? 2 : 1); ++h)
#pragma unroll
            for (int q = 0; q < CPL / 4; ++q) {
              const int ch = h * 128 + g * CPL + 4 * q;
              const float4 a = mean(nt, h * 8 + 2 * q, e);
              if (whole) store_row<BF16>(p, w.r, w.hk, w.tile * R + row, ch, a);
              else *reinterpret_cast<float4*>(slot + (size_t)row * DH + ch) = a;
            }
          if (!whole && g == 0) {
            slot[R * DH + row] = m[nt][e];
            slot[R * DH + R + row] = l[nt][e];
          }
        }
    }
    // rounds of RPR rows
    for (int r0 = 0; !WARPS && r0 < rows; r0 += RPR) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = nt * 8 + 2 * t + e;  // lane (g, t): rows 2t, 2t + 1, channels g * CPL ..
          if (row >= r0 && row < r0 + RPR && row < rows) {
#pragma unroll
            for (int h = 0; h < (DH == 256 ? 2 : 1); ++h) {
              float* d = mbuf + ((size_t)warp * RPR + row - r0) * DH + h * 128 + g * CPL;
#pragma unroll
              for (int q = 0; q < CPL / 4; ++q) *reinterpret_cast<float4*>(d + 4 * q) = mean(nt, h * 8 + 2 * q, e);
            }
          }
        }
      __syncthreads();
      for (int i = tid; i < min(RPR, rows - r0) * DH / 4; i += 32 * NCW) {
        const int row = i / (DH / 4), ch = (i % (DH / 4)) * 4, rr = r0 + row;
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int k = 0; k < NCW; ++k) M = fmaxf(M, s_m[k][rr]);
        // the warps with keys: those with weights (a warp whose scores are all NaN is one: fmaxf
        // leaves its maximum at -inf, and its sums have to arrive)
        float wt[NCW];
#pragma unroll
        for (int k = 0; k < NCW; ++k) {
          wt[k] = s_l[k][rr];
          if (wt[k] != 0.f) wt[k] *= ex2(s_m[k][rr] - M);
          L += wt[k];
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NCW; ++k) {
          if (wt[k] == 0.f) continue;
          const float f = wt[k] * inv;
          const float4 x = *reinterpret_cast<const float4*>(mbuf + ((size_t)k * RPR + row) * DH + ch);
          a.x += x.x * f;
          a.y += x.y * f;
          a.z += x.z * f;
          a.w += x.w * f;
        }
        if (whole) {
          store_row<BF16>(p, w.r, w.hk, w.tile * R + rr, ch, a);
        } else {
          *reinterpret_cast<float4*>(slot + (size_t)rr * DH + ch) = a;
          if (ch == 0) {
            slot[R * DH + rr] = M;
            slot[R * DH + R + rr] = L;
          }
        }
      }
      __syncthreads();  // the buffer is free again
    }
    if (!whole) {
      // the tile's parts lie with teams ta .. tb, the first of which names its counter
      const int ta = team_of(C, nc, w.at + p.tile_cost), tb = team_of(C, nc, w.at + w.len(p) - 1), parts = tb - ta + 1;
      bool last;
      __threadfence();
      if constexpr (WARPS) {
        __syncwarp();
        unsigned old = 0;
        if (lane == 0) {
          old = atomicAdd(p.counters + ta, 1u);
          if (old == (unsigned)(parts - 1)) p.counters[ta] = 0;
        }
        last = __shfl_sync(0xffffffffu, old, 0) == (unsigned)(parts - 1);
      } else {
        __syncthreads();
        if (tid == 0) {
          s_last = atomicAdd(p.counters + ta, 1u) == (unsigned)(parts - 1);
          if (s_last) p.counters[ta] = 0;
        }
        __syncthreads();
        last = s_last;
      }
      if (last) {
        __threadfence();
        // team ta's part is the last of its line (slot 1), the others' the first of theirs
        auto part_of = [&](int i) { return p.slots + (size_t)(2 * (ta + i) + (i == 0 ? 1 : 0)) * p.slot_floats; };
        for (int i = WARPS ? lane : tid; i < rows * DH / 4; i += 32 * TEAM) {
          const int rr = i / (DH / 4), ch = (i % (DH / 4)) * 4;
          float M = -INFINITY, L = 0.f;
          for (int k0 = 0; k0 < parts; k0 += 4) {
            float mk[4], lk[4], top = M;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float* q = part_of(min(k0 + k, parts - 1)) + R * DH + rr;
              mk[k] = __ldcg(q);
              lk[k] = k0 + k < parts ? __ldcg(q + R) : 0.f;
              top = fmaxf(top, mk[k]);
            }
            L = L == 0.f ? 0.f : L * ex2(M - top);
#pragma unroll
            for (int k = 0; k < 4; ++k) L += lk[k] == 0.f ? 0.f : lk[k] * ex2(mk[k] - top);
            M = top;
          }
          const float inv = L == 0.f ? 0.f : 1.f / L;
          float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int k = 0; k < parts; ++k) {
            const float* q = part_of(k);
            const float mk = __ldcg(q + R * DH + rr), lk = __ldcg(q + R * DH + R + rr);
            const float4 x = __ldcg(reinterpret_cast<const float4*>(q + (size_t)rr * DH + ch));
            const float f = lk == 0.f ? 0.f : lk * ex2(mk - M) * inv;
            a.x += x.x * f;
            a.y += x.y * f;
            a.z += x.z * f;
            a.w += x.w * f;
          }
          store_row<BF16>(p, w.r, w.hk, w.tile * R + rr, ch, a);
        }
      }
    }
    if (w.at + w.len(p) >= u1) break;
    w.next(p);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// ------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------

// Query rows of a tile of k_kv8_attn_split: 8 or 16 (8 where a row is 256 wide: 16 rows of
// sums would not fit the registers).
static int split_rows(int64_t dh, int64_t rows) { return rows <= 8 || dh == 256 ? 8 : 16; }

static size_t split_slot_floats(int64_t dh, int64_t rows) { return (size_t)split_rows(dh, rows) * (dh + 2); }

size_t kv8_attention_ws_size(int64_t dh, int64_t rows) {
  size_t slots = (size_t)2 * kMaxTeams * split_slot_floats(dh, rows);
  if (prompt_takes(true, dh, rows, INT64_MAX)) slots = std::max(slots, (size_t)2 * kMaxCtas * prompt_slot_floats(dh));
  return round_up((size_t)kMaxTeams * 4, kAlign) + round_up(slots * 4, kAlign);
}

using SplitKernel = void (*)(const AttnParams);
struct SplitPick {
  SplitKernel kern;
  int threads;
  size_t smem;
};

template <bool BF16, bool E4M3, int DH, int NT>
static SplitPick split_pick(bool warps) {
  using Sh = SplitShape<BF16, DH, NT>;
  return {warps ? k_kv8_attn_split<BF16, E4M3, DH, NT, true> : k_kv8_attn_split<BF16, E4M3, DH, NT, false>, Sh::THREADS, Sh::SMEM};
}

template <bool BF16, bool E4M3>
static SplitPick split_pick(int64_t dh, int rows, bool warps) {
  if (dh == 64) return rows == 8 ? split_pick<BF16, E4M3, 64, 1>(warps) : split_pick<BF16, E4M3, 64, 2>(warps);
  if (dh == 128) return rows == 8 ? split_pick<BF16, E4M3, 128, 1>(warps) : split_pick<BF16, E4M3, 128, 2>(warps);
  return split_pick<BF16, E4M3, 256, 1>(warps);
}

static wina_status_t launch_split(AttnParams& p, bool bf16, int64_t rows, cudaStream_t s) {
  const int64_t dh = p.c.dh;
  const int R = split_rows(dh, rows);
  p.slot_floats = (int)split_slot_floats(dh, rows);
  const int sms = device_sm_count();
  if (sms < 1) return WINA_ERR_CUDA;
  const int64_t tiles = p.B * p.c.heads * ((rows + R - 1) / R);
  p.tiles = (int)std::min<int64_t>(tiles, INT32_MAX);
  // Two tiles or more to an SM: each warp works for itself, so that the tiles' fixed costs (4 us:
  // queries, one dependent pass, joining) run side by side; fewer: a CTA's warps share a tile.
  // Measured (32 / 8 heads of 128): 512 tiles of 10 K keys 219 us against 232 us by CTAs, 2064
  // tiles of 100 keys 42 against 98; 128 tiles of 9 K keys 72 us against 63, 8 of 16 K 149
  // against 22.
  const bool warps = tiles >= 2 * sms;
  // A tile's fixed cost in chunks: 6 us where a CTA's warps wait for one another, against 0.18 us
  // a chunk (16 ragged sequences: 44.5 us with 16, 39.2 with 22, 37.3 with 30); none where no CTA
  // has parts of two tiles anyway.
  p.tile_cost = warps ? 2 : tiles * 2 <= sms ? 0 : 32;
  const bool e4 = p.c.format == KV8_E4M3;
  const SplitPick k = bf16 ? (e4 ? split_pick<true, true>(dh, R, warps) : split_pick<true, false>(dh, R, warps))
                           : (e4 ? split_pick<false, true>(dh, R, warps) : split_pick<false, false>(dh, R, warps));
  const size_t smem = k.smem + round_up((size_t)pre_entries(p.B) * 4, 16);
  return cuda_status(launch_kernel(k.kern, dim3((unsigned)std::min(sms, kMaxCtas)), dim3((unsigned)k.threads), smem, s, false, p));
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
  if (T == 0) return WINA_OK;
  if (!q || !table || !kv_len || !out || !ws || !aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) ||
      !aligned(table, 4) || !aligned(kv_len, 4) || !aligned(cu_q, 4))
    return WINA_ERR_INVALID_ARG;
  if (ws_bytes < kv8_attention_ws_size(cache->dh, max_q * (Hq / cache->heads))) return WINA_ERR_WORKSPACE;
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
  p.slots = reinterpret_cast<float*>((char*)ws + round_up((size_t)kMaxTeams * 4, kAlign));
  const int64_t rows = max_q * (Hq / cache->heads);
  if (prompt_takes(qdt == WINA_BF16, cache->dh, rows, T * Hq)) return launch_prompt(p, (cudaStream_t)stream);
  return launch_split(p, qdt == WINA_BF16, rows, (cudaStream_t)stream);
}
