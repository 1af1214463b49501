// Attention of single tokens and of trees of drafted tokens over the
// microscaled KV cache.
//
// Rows: the query rows of a request that read one KV head, row = node * G +
// query head in the group; a chunk is what one warp takes together (MxRows).  A
// unit is (request, KV head, chunk); the tiles of all units form one list, and
// every warp of the grid takes the same number (or one more) of consecutive
// tiles of it, whatever unit they belong to: ragged batches and single long
// contexts fill the machine alike.  A warp computes alone: one warp of its block
// fills its ring with TMA bulk copies, its softmax state and sums stay in its
// registers, and a unit that it holds whole is finished there.  A unit that
// spans warps leaves one partial result per warp; the merge kernels add them up.
//
// Scores: A = 16 query rows x 16 channels, B = the codes of 8 tokens as fp16
// (exact), fp32 sums per block of 32 channels, times the block's scale in
// fp32.  The C fragment then holds, in lane (g, c), row g and tokens 4c..4c+3,
// which is the B operand of the second product: O^T += V^T (16 channels x 16
// tokens, codes as fp16) x P^T.  No exchange between lanes is needed.
//
// A value's scale goes onto the weight: w = 2^(x + e - M), x the score in
// log2 units, e the scale's exponent, M a reference per row and block of
// channels, so that the largest weights of each block use fp16's upper range
// whatever the scales are.  M and the row's own reference m are raised only
// when a score exceeds m by 10 or a weight exceeds 2^15, which after the first
// tiles is rare; the sums are rescaled then, and the largest weight stands at
// 2^8: halfway between fp16's top and where its 11 bits begin to run out, at
// 2^-22 of the largest weight.
//
// With bf16 queries and outputs the weights are one fp16 term: their 11 bits are 3
// more than the output keeps, and the error against 64 bits is that of the
// output's rounding (0.00165 relative; 0.00164 with fp32 weights).  With fp32 in or
// out there are two terms.
//
// Bounds (16 heads x 128; one call, inputs not in L2; B200s differ): 32 requests of
// 6-18K tokens, e4m3, trees of up to 8: 250 to 275 us, 5.3 to 5.8 TB/s, 81 to 89% of
// a copy.  One row each, e2m1: 156 to 168 us, 4.8 to 5.1 TB/s: 410 instructions per tile
// of 32 tokens, tensor pipe 42%, issue slots 52%, the slowest SM 10% behind the
// median.  One token over 32K, e4m3: 34 us against 21 of bytes: 3 us until the
// lengths, the page and the first tile have come one after another, 4 us for the
// merge, and shares of only 10 tiles per warp.  mx_attn_kernel<128, e4m3, 0, 1, 1> keeps
// its 12 warps at the price of 120 bytes of spills.
#include <cmath>

#include "mx_attn.cuh"

namespace loopvq {
namespace {

constexpr uint32_t kIdleLimit = 1u << 23;   // polls of the feeding warp, a third of a second at least

// One block per SM: kWarps warps that compute and one that feeds them.  Each
// has a ring of kStages slots (a tile of K and its tile of V); 100 to 200 KB per
// SM are on their way at a time.  With the feeding warp that is 16 warps of up to
// 128 registers, 12 of 168, or 8 of 255.
template <int D, int FMT, int NARROW, int NT>
struct MxRing {
  static constexpr int kSlot = 2 * MxTile<D, FMT>::kBytes;
  static constexpr int kWarps = NARROW ? (kSlot > 8000 ? 11 : 15) : NT == 1 ? 11 : 7;
  static constexpr int kFit = 212 * 1024 / (kWarps * kSlot);
  static constexpr int kStages = kFit < 4 ? kFit : 4;
  static constexpr int kBytes = kWarps * kStages * kSlot;
  static_assert(kStages >= 2, "one slot is read while the next arrives");
};

// d = a (16 x 16) b (16 x 8) + c
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// Rows of a request that one warp takes together, as NT groups of columns of
// the second product.
//   NARROW 0: a column is a query row; a lane goes through all blocks.
//   NARROW 1: a column is a (query row, block of channels), so that a lane
//             scales, exponentiates and packs weights for one block only.
//   NARROW 2: a column is a (half of the tile, query row, block): one such
//             pass covers both halves.  The halves are summed at the end as
//             two parts of a split context.
// Measured on 32 requests of 6-18K tokens, one row each, e2m1, D = 128, replayed in a
// graph: kind 0 249 us, kind 1 181 us, kind 2 161 us (149 since a warp of its own
// feeds the rings).
template <int D, int NARROW>
struct MxRows {
  static constexpr int kPerGroup = NARROW ? 8 / (D / kMxBlock) / NARROW : 8;
};

// TERMS: fp16 terms of queries and weights; EXACT: the cap's tanh (kFastCap).
template <int D, int FMT, int NARROW, int TERMS, int NT, bool EXACT>
__global__ void __launch_bounds__((MxRing<D, FMT, NARROW, NT>::kWarps + 1) * 32, 1) mx_attn_kernel(const MxAttnParams p) {
  using Tile = MxTile<D, FMT>;
  using Ring = MxRing<D, FMT, NARROW, NT>;
  constexpr int NB = Tile::kBlocks, S = Ring::kStages, W = Ring::kWarps;
  constexpr int RPG = MxRows<D, NARROW>::kPerGroup, CHUNK = RPG * NT;
  constexpr int MT = TERMS == 2 ? NT : (NT + 1) / 2;   // 16-row operands of the score product
  constexpr bool kBoth = TERMS == 2 || NT > 1;         // both halves of the 16 rows are used
  constexpr int NW = NARROW ? 1 : NB;                  // blocks that a lane weighs
  extern __shared__ __align__(128) uint8_t sm_ring[];
  __shared__ __align__(8) uint64_t full[W][S], empty[W][S];
  __shared__ __align__(16) float sm_scale[NARROW ? 1 : W][2][NARROW ? 4 : 32 * NB];   // of the tile: K, V
  __shared__ MxCursor sm_start[W];
  __shared__ int sm_count[W];
  __shared__ uint32_t sm_bad[W];   // bit per slot: its tile's page is not in the pool
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  constexpr int SUBS = NARROW == 2 ? 2 : 1;            // halves of a tile that are in flight together
  const int gb = NARROW ? g % NB : 0;                  // this lane's block,
  const int gr = NARROW ? g / NB % RPG : g;            // row in a group,
  const int half = NARROW == 2 ? g >> 2 : 0;           // half of the tile (NARROW 2)
  mx_begin();
  const int n_warps = p.n_workers, wid = blockIdx.x * W + warp;

  // each warp's share of the list: `extra` warps take one tile more than the others
  int64_t share = 0, begin = 0;
  int extra = 0, count = 0;
  MxCursor cc = {};
  if (warp < W) {
    int u0 = 0, t0 = 0;
    if (lane < p.L.batch) u0 = mx_units<CHUNK>(p, lane, &t0);
    int64_t total = (int64_t)u0 * t0;
    for (int r = lane + 32; r < p.L.batch; r += 32) {
      int tiles;
      const int units = mx_units<CHUNK>(p, r, &tiles);
      total += (int64_t)units * tiles;
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
    share = total / n_warps;
    extra = (int)(total % n_warps);
    begin = wid * share + min(wid, extra);
    count = (int)share + (wid < extra);
    if (count) cc = mx_seek<CHUNK>(p, begin, u0, t0, lane);
    if (lane == 0) {
      p.headers[wid] = make_int4(0, 0, 0, 0);
      sm_start[warp] = cc;
      sm_count[warp] = count;
      sm_bad[warp] = 0;
      for (int i = 0; i < S; ++i) {
        mbar_init(smem_u32(&full[warp][i]), 1);
        mbar_init(smem_u32(&empty[warp][i]), 1);
      }
      fence_mbar_init();
    }
  }
  __syncthreads();

  if (warp == W) {   // the feeding warp: lane w fills the ring of warp w
    const int n = lane < W ? sm_count[lane] : 0;
    if (n == 0) return;
    MxCursor pc = sm_start[lane];
    const int per = p.L.page_tokens / kMxTile;
    int page = pc.t / per, in_page = pc.t % per, slot = 0;
    uint32_t phase = 1, idle = 0;   // a wait for the phase before the first does not block
    int64_t head = (int64_t)(pc.u / (pc.units / p.H)) * p.L.pool_tiles;
    int id = ld_once(p.L.pages + (int64_t)pc.r * p.L.max_pages + page);
    const uint32_t ring = smem_u32(sm_ring) + lane * S * Ring::kSlot;
    for (int i = 0; i < n;) {
      if (!mbar_test(smem_u32(&empty[lane][slot]), phase)) {
        if (++idle > kIdleLimit) {   // the warp has given up: nothing of this ring is read any more
          set_fault(p.fault, LOOPVQ_FAULT_TIMEOUT);
          return;
        }
        __nanosleep(40);
        continue;
      }
      idle = 0;
      const uint32_t bar = smem_u32(&full[lane][slot]);
      if (id >= 0 && id < p.L.n_pages) {
        const int64_t at = (head + (int64_t)id * per + in_page) * Tile::kBytes;
        mbar_arrive_expect_tx(bar, 2 * Tile::kBytes);
        bulk_g2s(ring + slot * Ring::kSlot, p.pk + at, Tile::kBytes, bar);
        bulk_g2s(ring + slot * Ring::kSlot + Tile::kBytes, p.pv + at, Tile::kBytes, bar);
      } else {
        set_fault(p.fault, LOOPVQ_FAULT_POOL_RANGE);
        atomicOr(&sm_bad[lane], 1u << slot);   // before the arrival that publishes it
        mbar_arrive(bar);
      }
      if (++slot == S) {
        slot = 0;
        phase ^= 1;
      }
      if (++i == n) break;
      if (++pc.t == pc.tiles) {
        mx_next_unit<CHUNK>(p, &pc);
        page = in_page = 0;
        head = (int64_t)(pc.u / (pc.units / p.H)) * p.L.pool_tiles;
        id = ld_once(p.L.pages + (int64_t)pc.r * p.L.max_pages);
      } else if (++in_page == per) {
        in_page = 0;
        ++page;
        id = ld_once(p.L.pages + (int64_t)pc.r * p.L.max_pages + page);
      }
    }
    return;
  }

  const uint8_t* const ring = sm_ring + warp * S * Ring::kSlot;
  int done = 0, slot = 0;
  uint32_t phase = 0;
  bool lost = false;
  while (done < count && !lost) {
    // ------------------------------------------------ a unit, or the part of it in this share
    MxReq rq = {};
    mx_request(p.L, cc.r, &rq, nullptr);
    const int chunks = cc.units / p.H, h = cc.u / chunks, rho0 = (cc.u - h * chunks) * CHUNK;
    const int rows = max(0, min(CHUNK, rq.n * p.G - rho0));   // 0 if lengths change meanwhile
    const int first_tile = cc.t, n_tiles = min(cc.tiles - cc.t, count - done);
    const uint64_t all_new = rq.n >= 64 ? ~0ull : (1ull << rq.n) - 1;

    // query rows
    float v[NT][NW][8] = {};
    float f[NT], slope[NT];
    uint64_t sees[NT];
    int pos_q[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int rho = rho0 + RPG * i + gr;
      slope[i] = 0.f;
      sees[i] = 0;
      pos_q[i] = 0;
      if (rho < rq.n * p.G) {
        const int node = rho / p.G, hq = h * p.G + rho % p.G;
        const int64_t at = (int64_t)(rq.row0 + node) * p.qn + (int64_t)hq * p.qh + 32 * gb + 8 * c;
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          if (p.q_bf16) load_query<__nv_bfloat16>(p.q, at + 32 * b, p.q_vec, v[i][b]);
          else load_query<float>(p.q, at + 32 * b, p.q_vec, v[i][b]);
        }
        sees[i] = (p.tree_mask ? ld_once(p.tree_mask + rq.row0 + node) : (2ull << node) - 1) & all_new;
        pos_q[i] = rq.base + __popcll(sees[i] & ~(1ull << node));
        if (p.slopes) slope[i] = ld_once(p.slopes + hq) * kLog2e;
      }
    }
    // scaled by a power of two (NARROW: of each block) to a largest magnitude in
    // [2^14, 2^15), as fp16 (TERMS = 2: and the rest)
    uint32_t qa[MT][NB][2][4] = {};
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float mx = 0.f;
#pragma unroll
      for (int b = 0; b < NW; ++b)
#pragma unroll
        for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(v[i][b][k]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = max((int)(__float_as_uint(mx) >> 23), 1) - 127;
      const int k2 = min(14 - ex, 120);
      const float up = __uint_as_float((uint32_t)(127 + k2) << 23), down = __uint_as_float((uint32_t)(129 - k2) << 23);
      f[i] = p.scale * down;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int vb = NARROW ? 0 : b;
          const bool has = !NARROW || gb == b;   // NARROW: a row of block b is 0 elsewhere
          const float x0 = v[i][vb][2 * k] * up, x1 = v[i][vb][2 * k + 1] * up;
          const uint32_t hi = pack_f16(x0, x1);
          // pair k: channels 8c + 2k, 8c + 2k + 1: product k/2, upper half of its 16 channels if k is odd
          if constexpr (TERMS == 1) {
            qa[i / 2][b][k >> 1][(k & 1) * 2 + (i & 1)] = has ? hi : 0u;
          } else {
            const float2 b2 = unpack_f16(hi);
            qa[i][b][k >> 1][(k & 1) * 2] = has ? hi : 0u;
            qa[i][b][k >> 1][(k & 1) * 2 + 1] = has ? pack_f16(x0 - b2.x, x1 - b2.y) : 0u;
          }
        }
    }

    float m[NT], l[NT], M[NT][NW], rs[NT][NW], o[NW][2][NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int b = 0; b < NW; ++b) {
        M[i][b] = -INFINITY;
        rs[i][b] = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[b][0][i][k] = o[b][1][i][k] = 0.f;
      }
    }

    for (int it = 0; it < n_tiles; ++it) {
      const bool got = mbar_wait_bounded(smem_u32(&full[warp][slot]), phase);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) set_fault(p.fault, LOOPVQ_FAULT_TIMEOUT);
        lost = true;
        break;
      }
      const uint8_t* sk = ring + slot * Ring::kSlot;
      const uint8_t* sv = sk + Tile::kBytes;
      const int tok0 = (first_tile + it) * kMxTile;
      const bool edge = tok0 + kMxTile > rq.base;
      const uint32_t bad = *reinterpret_cast<volatile uint32_t*>(&sm_bad[warp]);
      if (!(bad >> slot & 1)) {
        if constexpr (!NARROW) {   // the tile's scales as fp32, once for all rows
          if (lane < 8 * NB) {
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t w = reinterpret_cast<const uint32_t*>((kv ? sv : sk) + Tile::kScaleOff)[lane];
              reinterpret_cast<float4*>(sm_scale[warp][kv])[lane] =
                  make_float4(scale_f32(w, 0), scale_f32(w, 1), scale_f32(w, 2), scale_f32(w, 3));
            }
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int sub = 0; sub < 2; sub += SUBS) {
          const int quad = (sub + half) * 4 + c;   // this lane's tokens: 4 * quad ..
          // ---- scores
          float s[SUBS][MT][2][4] = {};
          float2 ksc[2];   // NARROW: this lane's block and tokens
          if constexpr (NARROW) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(sk + mx_scale_off<D, FMT>(quad, gb));
            ksc[0] = make_float2(scale_f32(w, 0), scale_f32(w, 1));
            ksc[1] = make_float2(scale_f32(w, 2), scale_f32(w, 3));
          }
#pragma unroll
          for (int b = 0; b < NB; b += 2)
#pragma unroll
            for (int su = 0; su < SUBS; ++su) {
              uint32_t hc[2][2][4];   // [block][ab][pair]
              if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const uint4 w = *reinterpret_cast<const uint4*>(sk + mx_code_off<D, FMT>(sub + su, b + k, lane));
                  codes_e4m3(w.x, hc[k][0]);
                  codes_e4m3(w.y, hc[k][0] + 2);
                  codes_e4m3(w.z, hc[k][1]);
                  codes_e4m3(w.w, hc[k][1] + 2);
                }
              } else {
                const uint4 w = *reinterpret_cast<const uint4*>(sk + mx_code_off<D, FMT>(sub + su, b, lane));
                codes_e2m1(w.x, hc[0][0]);
                codes_e2m1(w.y, hc[0][1]);
                codes_e2m1(w.z, hc[1][0]);
                codes_e2m1(w.w, hc[1][1]);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float4 sc = {};
                if constexpr (!NARROW)
                  sc = reinterpret_cast<const float4*>(sm_scale[NARROW ? 0 : warp][0])[quad * NB + b + k];
#pragma unroll
                for (int ab = 0; ab < 2; ++ab) {
#pragma unroll
                  for (int i = 0; i < MT; ++i) {
                    const uint32_t(*a)[4] = qa[i][b + k];
                    if constexpr (NARROW) {
                      mma_f16(s[su][i][ab], a[0], hc[k][ab][0], hc[k][ab][1], s[su][i][ab]);
                      mma_f16(s[su][i][ab], a[1], hc[k][ab][2], hc[k][ab][3], s[su][i][ab]);
                    } else {
                      const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                      float d[4];
                      mma_f16(d, a[0], hc[k][ab][0], hc[k][ab][1], zero);
                      mma_f16(d, a[1], hc[k][ab][2], hc[k][ab][3], d);
                      const float2 s2 = ab ? make_float2(sc.z, sc.w) : make_float2(sc.x, sc.y);
                      fma2(&s[su][i][ab][0], make_float2(d[0], d[1]), s2);
                      if constexpr (kBoth) fma2(&s[su][i][ab][2], make_float2(d[2], d[3]), s2);
                    }
                  }
                }
              }
            }
          // ---- in log2 units (up to the cap in natural ones), with cap, bias and mask: row gr of group i, tokens 4c + t
          const int pos = tok0 + 4 * quad;
          float x[NT][4];
          uint32_t hide = 0;   // bit 4i + t: not seen
#pragma unroll
          for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int ab = 0; ab < 2; ++ab) {
              float2 y;
              if constexpr (NARROW == 2) {   // rows g and g ^ 4 are the same query and block: this lane keeps its half of the tile
                y = half ? make_float2(s[SUBS - 1][i / 2][ab][0], s[SUBS - 1][i / 2][ab][1])
                         : make_float2(s[0][i / 2][ab][0], s[0][i / 2][ab][1]);
                if constexpr (TERMS == 2) {
                  y.x += half ? s[SUBS - 1][i / 2][ab][2] : s[0][i / 2][ab][2];
                  y.y += half ? s[SUBS - 1][i / 2][ab][3] : s[0][i / 2][ab][3];
                }
              } else if constexpr (TERMS == 2) {
                y = make_float2(s[0][i % MT][ab][0] + s[0][i % MT][ab][2], s[0][i % MT][ab][1] + s[0][i % MT][ab][3]);
              } else {
                y = make_float2(s[0][i / 2][ab][2 * (i & 1)], s[0][i / 2][ab][2 * (i & 1) + 1]);
              }
              y = mul2(y, make_float2(f[i], f[i]));
              if constexpr (NARROW) {   // scaled, and summed over the blocks
                y = mul2(y, ksc[ab]);
#pragma unroll
                for (int d = 4; d < 4 * NB; d <<= 1) {
                  y.x += __shfl_xor_sync(0xffffffffu, y.x, d);
                  y.y += __shfl_xor_sync(0xffffffffu, y.y, d);
                }
              }
              x[i][2 * ab] = y.x;
              x[i][2 * ab + 1] = y.y;
            }
          }
          if (p.softcap > 0.f) {
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int t = 0; t < 4; ++t)
                x[i][t] = EXACT ? capped(x[i][t], p.softcap, p.inv_cap) : capped_fast(x[i][t], p.softcap, p.inv_cap2);
          }
          if (p.slopes || edge) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int j = pos + t - rq.base;   // >= 0: a new token
              int at = pos + t;
              if (p.slopes && j >= 0 && j < rq.n) {
                const uint64_t its = p.tree_mask ? ld_once(p.tree_mask + rq.row0 + j) & all_new : (2ull << j) - 1;
                at = rq.base + __popcll(its & ~(1ull << j));
              }
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                if (p.slopes) x[i][t] -= slope[i] * (float)(pos_q[i] - at);
                const bool see = j < 0 || (j < rq.n && (sees[i] >> j & 1));
                if (!see) {
                  x[i][t] = -INFINITY;
                  hide |= 1u << (4 * i + t);
                }
              }
            }
          }
          // ---- weights
          float4 vsc[NW];
          if constexpr (NARROW) {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(sv + mx_scale_off<D, FMT>(quad, gb));
            vsc[0] = make_float4(scale_f32(w, 0), scale_f32(w, 1), scale_f32(w, 2), scale_f32(w, 3));
          } else {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              vsc[b] = reinterpret_cast<const float4*>(sm_scale[NARROW ? 0 : warp][1])[quad * NB + b];
          }
          uint32_t pw[NT][NW][TERMS][2];
          float pr[NT];
          auto weights = [&]() {
            bool over = false;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              const float mi = m[i] == -INFINITY ? 0.f : m[i];
              float e[4];
#pragma unroll
              for (int t = 0; t < 4; ++t) e[t] = ex2(x[i][t] - mi);
              pr[i] = (e[0] + e[1]) + (e[2] + e[3]);
              over |= fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3])) > m[i] + kScoreSlack;
              float wm = 0.f;
#pragma unroll
              for (int b = 0; b < NW; ++b) {
                float2 w[2] = {mul2(make_float2(e[0], e[1]), make_float2(vsc[b].x, vsc[b].y)),
                               mul2(make_float2(e[2], e[3]), make_float2(vsc[b].z, vsc[b].w))};
                w[0] = mul2(w[0], make_float2(rs[i][b], rs[i][b]));
                w[1] = mul2(w[1], make_float2(rs[i][b], rs[i][b]));
                if (edge) {   // 0 times the infinity that marks a block of NaN
                  if (hide >> (4 * i) & 1) w[0].x = 0.f;
                  if (hide >> (4 * i) & 2) w[0].y = 0.f;
                  if (hide >> (4 * i) & 4) w[1].x = 0.f;
                  if (hide >> (4 * i) & 8) w[1].y = 0.f;
                }
                wm = fmaxf(wm, fmaxf(fmaxf(w[0].x, w[0].y), fmaxf(w[1].x, w[1].y)));
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  pw[i][b][0][k] = pack_f16(w[k].x, w[k].y);
                  if constexpr (TERMS == 2) {
                    const float2 hi = unpack_f16(pw[i][b][0][k]);
                    pw[i][b][1][k] = pack_f16(w[k].x - hi.x, w[k].y - hi.y);
                  }
                }
              }
              over |= wm > kWeightMax;
            }
            return over;
          };
          // the first tile sets the references, later ones seldom raise them
          if ((it == 0 && sub == 0) || __any_sync(0xffffffffu, weights())) {
            {
              // raise the references to what has been seen, and bring the sums to them
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                float mx = fmaxf(fmaxf(x[i][0], x[i][1]), fmaxf(x[i][2], x[i][3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[i], mx);
                if (m[i] != -INFINITY) l[i] *= ex2(m[i] - mn);
                m[i] = mn;
#pragma unroll
                for (int b = 0; b < NW; ++b) {
                  // scales are powers of two: their exponents, 128 for the infinity that marks NaN
                  const float ve[4] = {vsc[b].x, vsc[b].y, vsc[b].z, vsc[b].w};
                  float bm = -INFINITY;
#pragma unroll
                  for (int t = 0; t < 4; ++t) bm = fmaxf(bm, x[i][t] + (float)((int)(__float_as_uint(ve[t]) >> 23) - 127));
                  bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 1));
                  bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 2));
                  const float Mn = fmaxf(M[i][b], bm - kWeightExp);
                  const float fb = M[i][b] == -INFINITY ? 0.f : ex2(M[i][b] - Mn);
                  M[i][b] = Mn;
                  rs[i][b] = Mn == -INFINITY ? 0.f : ex2(mn - Mn);
#pragma unroll
                  for (int k = 0; k < 2; ++k) {
                    const float fc = __shfl_sync(0xffffffffu, fb, (2 * c + k) * 4);
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                      o[b][a][i][k] *= fc;
                      o[b][a][i][2 + k] *= fc;
                    }
                  }
                }
              }
            }
            weights();
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) l[i] += pr[i];
          // ---- values
#pragma unroll
          for (int b = 0; b < NB; b += 2)
#pragma unroll
            for (int su = 0; su < SUBS; ++su) {
              uint32_t hv[2][4][2];   // [block][channel j][token pair]
              if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint4 w = *reinterpret_cast<const uint4*>(sv + mx_code_off<D, FMT>(sub + su, b + k, lane));
                  if (edge) {
                    w.x = drop_nan_codes(w.x);
                    w.y = drop_nan_codes(w.y);
                    w.z = drop_nan_codes(w.z);
                    w.w = drop_nan_codes(w.w);
                  }
                  codes_e4m3(w.x, hv[k][0]);
                  codes_e4m3(w.y, hv[k][1]);
                  codes_e4m3(w.z, hv[k][2]);
                  codes_e4m3(w.w, hv[k][3]);
                }
              } else {
                const uint4 w = *reinterpret_cast<const uint4*>(sv + mx_code_off<D, FMT>(sub + su, b, lane));
                codes_e2m1(w.x, hv[0][0]);
                codes_e2m1(w.y, hv[0][2]);
                codes_e2m1(w.z, hv[1][0]);
                codes_e2m1(w.w, hv[1][2]);
              }
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int wb = NARROW ? 0 : b + k;
                // NARROW: the columns of this block (and half of the tile)
                const bool mine = !NARROW || (gb == b + k && (SUBS == 1 || half == su));
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                  const uint32_t va[4] = {hv[k][2 * a][0], hv[k][2 * a + 1][0], hv[k][2 * a][1], hv[k][2 * a + 1][1]};
#pragma unroll
                  for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < TERMS; ++e)
                      mma_f16(o[wb][a][i], va, mine ? pw[i][wb][e][0] : 0u, mine ? pw[i][wb][e][1] : 0u, o[wb][a][i]);
                }
              }
            }
        }
      }
      __syncwarp();   // every lane has read the slot
      if (lane == 0) {
        if (bad >> slot & 1) atomicAnd(&sm_bad[warp], ~(1u << slot));
        mbar_arrive(smem_u32(&empty[warp][slot]));
      }
      ++done;
      if (++slot == S) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (lost) break;

    // ------------------------------------------------ the unit's rows, or this warp's part of them
    const bool whole = first_tile == 0 && n_tiles == cc.tiles;
    float* part = p.partials + (size_t)(2 * wid + (first_tile == 0)) * CHUNK * (D + 4);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float ls = l[i], mt = m[i];
      ls += __shfl_xor_sync(0xffffffffu, ls, 1);
      ls += __shfl_xor_sync(0xffffffffu, ls, 2);
      const float own = ls;
      if constexpr (NARROW == 2) {   // the halves: relative to the larger reference
        const float lo = __shfl_xor_sync(0xffffffffu, ls, 16), mo = __shfl_xor_sync(0xffffffffu, mt, 16);
        mt = fmaxf(m[i], mo);
        ls = (m[i] == -INFINITY ? ls : ls * ex2(m[i] - mt)) + (mo == -INFINITY ? lo : lo * ex2(mo - mt));
      }
      const int mine = RPG * i + gr;
      const float lse = ls == 0.f ? -INFINITY : (mt + log2f(ls)) * kLn2;
      if (c == 0 && gb == 0 && half == 0 && mine < rows) {
        const int rho = rho0 + mine;
        if (!whole) {
          *reinterpret_cast<float2*>(part + mine * (D + 4) + D) = make_float2(mt, ls);
        } else if (p.lse) {
          p.lse[(int64_t)(rq.row0 + rho / p.G) * p.Hq + h * p.G + rho % p.G] = lse;
        }
      }
      const float inv = whole ? (ls == 0.f ? 0.f : 1.f / ls) : 1.f;
      float fb[NW];   // a row that saw only NaN has no M: its l is NaN
#pragma unroll
      for (int b = 0; b < NW; ++b) fb[b] = M[i][b] == -INFINITY ? own : ex2(M[i][b] - mt) * inv;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = 2 * c + k;
        const int row = RPG * i + (NARROW ? col / NB % RPG : col), rho = rho0 + row;
        const int64_t at = ((int64_t)(rq.row0 + rho / p.G) * p.Hq + h * p.G + rho % p.G) * D;
#pragma unroll
        for (int b = 0; b < NW; ++b) {
          const float fc = __shfl_sync(0xffffffffu, fb[b], col * 4);
          const int ch = 32 * (NARROW ? col % NB : b) + 4 * g;
          float4 y = make_float4(o[b][0][i][k] * fc, o[b][0][i][2 + k] * fc, o[b][1][i][k] * fc, o[b][1][i][2 + k] * fc);
          if constexpr (NARROW == 2) {
            y.x += __shfl_xor_sync(0xffffffffu, y.x, 2);
            y.y += __shfl_xor_sync(0xffffffffu, y.y, 2);
            y.z += __shfl_xor_sync(0xffffffffu, y.z, 2);
            y.w += __shfl_xor_sync(0xffffffffu, y.w, 2);
            if (c >= 2) continue;
          }
          if (row >= rows) continue;
          if (!whole) {
            *reinterpret_cast<float4*>(part + row * (D + 4) + ch) = y;
          } else if (p.out_bf16) {
            const __nv_bfloat162 z0 = __floats2bfloat162_rn(y.x, y.y), z1 = __floats2bfloat162_rn(y.z, y.w);
            *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at + ch) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&z0), *reinterpret_cast<const uint32_t*>(&z1));
          } else {
            *reinterpret_cast<float4*>(reinterpret_cast<float*>(p.out) + at + ch) = y;
          }
        }
      }
    }
    if (first_tile == 0 && !whole && lane == 0) {
      // the warps after this one that hold the unit's other tiles
      const int64_t last = begin + done - n_tiles + cc.tiles - 1, longer = (int64_t)extra * (share + 1);
      const int64_t owner = last < longer ? last / (share + 1) : extra + (last - longer) / share;
      p.headers[wid] = make_int4((int)(owner - wid), rq.row0, h, rho0 << 8 | rows);
    }
    if (done < count) mx_next_unit<CHUNK>(p, &cc);
  }
  if (lost) {   // copies that are still on their way end before the block does
    for (int i = 0; i < S; ++i) {
      mbar_wait_bounded(smem_u32(&full[warp][slot]), phase);
      if (++slot == S) {
        slot = 0;
        phase ^= 1;
      }
    }
  }
}

// Adds up the partial results of units.  Block (x, y) takes the units that
// start in warps 4 x .. 4 x + 3 of the attention kernel and go on in warps after
// them, rows y, y + gridDim.y, ..  The references and sums of all parts
// are in shared memory before the first row is read, so that the rows' loads
// wait for nothing but memory; eight warps share the parts of a row.
// o += f * part, this lane's channels.
template <int N>
__device__ __forceinline__ void add_part(const float* part, int lane, float f, float* o) {
  if constexpr (N == 4) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(part) + lane);
    o[0] = fmaf(v.x, f, o[0]);
    o[1] = fmaf(v.y, f, o[1]);
    o[2] = fmaf(v.z, f, o[2]);
    o[3] = fmaf(v.w, f, o[3]);
  } else {
    const float2 v = __ldcg(reinterpret_cast<const float2*>(part) + lane);
    o[0] = fmaf(v.x, f, o[0]);
    o[1] = fmaf(v.y, f, o[1]);
  }
}
constexpr int kMergeWarps = 8, kMergeParts = 512, kMergeHeads = 4;
template <int D, int CHUNK>
__global__ void __launch_bounds__(kMergeWarps * 32) mx_merge_kernel(const MxAttnParams p) {
  constexpr int kCh = D / 32;   // channels of a lane
  __shared__ float sm_o[kMergeWarps][D];
  __shared__ float sm_f[kMergeParts], sm_l[kMergeWarps], sm_m[kMergeWarps];
  mx_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int4 hds[kMergeHeads];
#pragma unroll
  for (int i = 0; i < kMergeHeads; ++i) {
    const int w = blockIdx.x * kMergeHeads + i;
    hds[i] = w < p.n_workers ? __ldcg(p.headers + w) : make_int4(0, 0, 0, 0);
  }
#pragma unroll 1
  for (int i = 0; i < kMergeHeads; ++i) {
    const int4 hd = i == 0 ? hds[0] : i == 1 ? hds[1] : i == 2 ? hds[2] : hds[3];
    const int w = blockIdx.x * kMergeHeads + i, rows = hd.x ? hd.w & 255 : 0, rho0 = hd.w >> 8;
    for (int row = blockIdx.y; row < rows; row += gridDim.y) {
      auto part = [&](int k) {   // slot 1 of warp w, slot 0 of the next ones
        return p.partials + ((size_t)(2 * (w + k) + (k == 0)) * CHUNK + row) * (D + 4);
      };
      float top = -INFINITY, ls = 0.f, o[kCh] = {};
      for (int k0 = 0; k0 <= hd.x; k0 += kMergeParts) {   // one turn unless there are very many parts
        const int n = min(kMergeParts, hd.x + 1 - k0);
        float mk[kMergeParts / (kMergeWarps * 32)], lk[kMergeParts / (kMergeWarps * 32)], mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < kMergeParts / (kMergeWarps * 32); ++e) {
          const int k = threadIdx.x + e * kMergeWarps * 32;
          const float2 v = k < n ? __ldcg(reinterpret_cast<const float2*>(part(k0 + k) + D)) : make_float2(-INFINITY, 0.f);
          mk[e] = v.x;
          lk[e] = v.y;
          mx = fmaxf(mx, v.x);
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        if (lane == 0) sm_m[warp] = mx;
        __syncthreads();
        float tn = top;
#pragma unroll
        for (int e = 0; e < kMergeWarps; ++e) tn = fmaxf(tn, sm_m[e]);
        const float m0 = tn == -INFINITY ? 0.f : tn, back = top == -INFINITY ? 0.f : ex2(top - m0);
        ls *= back;
#pragma unroll
        for (int e = 0; e < kCh; ++e) o[e] *= back;
#pragma unroll
        for (int e = 0; e < kMergeParts / (kMergeWarps * 32); ++e) {
          const float f = ex2(mk[e] - m0);
          sm_f[threadIdx.x + e * kMergeWarps * 32] = f;
          ls += lk[e] * f;
        }
        top = tn;
        __syncthreads();
#pragma unroll 4
        for (int k = warp; k < n; k += kMergeWarps) {
          add_part<kCh>(part(k0 + k), lane, sm_f[k], o);
        }
        __syncthreads();   // the next turn writes sm_f and sm_m
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      if (lane == 0) sm_l[warp] = ls;
#pragma unroll
      for (int e = 0; e < kCh; ++e) sm_o[warp][lane * kCh + e] = o[e];
      __syncthreads();
      float l = 0.f;
#pragma unroll
      for (int e = 0; e < kMergeWarps; ++e) l += sm_l[e];
      const int rho = rho0 + row, d = threadIdx.x;
      const int64_t at = (int64_t)(hd.y + rho / p.G) * p.Hq + hd.z * p.G + rho % p.G;
      if (d < D) {
        float y = 0.f;
#pragma unroll
        for (int e = 0; e < kMergeWarps; ++e) y += sm_o[e][d];
        y *= l == 0.f ? 0.f : 1.f / l;
        if (p.out_bf16) reinterpret_cast<__nv_bfloat16*>(p.out)[at * D + d] = __float2bfloat16_rn(y);
        else reinterpret_cast<float*>(p.out)[at * D + d] = y;
      }
      if (d == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
      __syncthreads();
    }
  }
}

// The same for chunks of many rows: a warp takes a row, 32 parts at a time.
template <int D, int CHUNK>
__global__ void __launch_bounds__(kMergeWarps * 32) mx_merge_rows_kernel(const MxAttnParams p) {
  constexpr int kCh = D / 32;
  mx_begin();
  const int lane = threadIdx.x & 31, row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5);
  const int w = blockIdx.x;
  const int4 hd = __ldcg(p.headers + w);
  if (hd.x == 0 || row >= (hd.w & 255)) return;
  auto part = [&](int k) { return p.partials + ((size_t)(2 * (w + k) + (k == 0)) * CHUNK + row) * (D + 4); };
  float top = -INFINITY, l = 0.f, o[kCh] = {};
  for (int k0 = 0; k0 <= hd.x; k0 += 32) {
    const float2 ml =
        k0 + lane <= hd.x ? __ldcg(reinterpret_cast<const float2*>(part(k0 + lane) + D)) : make_float2(-INFINITY, 0.f);
    float tn = fmaxf(top, ml.x);
#pragma unroll
    for (int d = 16; d; d >>= 1) tn = fmaxf(tn, __shfl_xor_sync(0xffffffffu, tn, d));
    const float m0 = tn == -INFINITY ? 0.f : tn, back = top == -INFINITY ? 0.f : ex2(top - m0), fl = ex2(ml.x - m0);
    l = l * back + ml.y * fl;
#pragma unroll
    for (int e = 0; e < kCh; ++e) o[e] *= back;
    const int n = min(32, hd.x + 1 - k0);
#pragma unroll 8
    for (int k = 0; k < n; ++k) add_part<kCh>(part(k0 + k), lane, __shfl_sync(0xffffffffu, fl, k), o);
    top = tn;
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const int rho = (hd.w >> 8) + row;
  const int64_t at = (int64_t)(hd.y + rho / p.G) * p.Hq + hd.z * p.G + rho % p.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < kCh; ++e) o[e] *= inv;
  if (p.out_bf16) {
#pragma unroll
    for (int e = 0; e < kCh; e += 2)
      reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at * D + lane * kCh)[e / 2] =
          __floats2bfloat162_rn(o[e], o[e + 1]);
  } else {
#pragma unroll
    for (int e = 0; e < kCh; ++e) reinterpret_cast<float*>(p.out)[at * D + lane * kCh + e] = o[e];
  }
  if (lane == 0 && p.lse) p.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

// More rows than this: mx_rows_kernel, whose time hardly depends on them.  16
// heads over 32K, D = 128, e4m3: 105 us; the warps' kernel 60 at 16 rows, 87 at 32,
// 117 at 48, 144 at 64.  D = 64: 91 to 93 us; 40 at 16, 75 at 48, 93 at 64.
template <int D>
constexpr int kRowsFrom = D == 128 ? 40 : 64;
// The variant of a call: columns per row, groups.
struct AttnVariant {
  int narrow, nt, chunk;
  int workers;   // of the largest launch, and in a block
  int per_block;
  bool rows;     // mx_rows_kernel
};
template <int D, int FMT>
AttnVariant attn_variant_t(int64_t rows, bool fine) {
  AttnVariant v;
  constexpr int kFew = MxRows<D, 1>::kPerGroup;
  v.narrow = rows <= kFew / 2 ? 2 : rows <= (fine ? kFew : 2 * kFew);
  const int per = v.narrow ? kFew / v.narrow : 8;
  v.nt = rows > per ? 2 : 1;
  v.chunk = per * v.nt;
  v.per_block = v.narrow == 2 ? MxRing<D, FMT, 2, 1>::kWarps
           : v.narrow    ? (v.nt == 2 ? MxRing<D, FMT, 1, 2>::kWarps : MxRing<D, FMT, 1, 1>::kWarps)
                         : (v.nt == 2 ? MxRing<D, FMT, 0, 2>::kWarps : MxRing<D, FMT, 0, 1>::kWarps);
  v.workers = device_sm_count() * v.per_block;
  v.rows = !fine && rows > kRowsFrom<D>;
  if (v.rows) {
    v.chunk = kMxRowsChunk;
    v.workers = mx_rows_workers();
    v.per_block = 1;
  }
  return v;
}
AttnVariant attn_variant(const loopvq_mx_desc* d, const loopvq_mx_layout* l, bool fine) {
  const int64_t rows = (int64_t)l->max_new * (d->n_heads_q / d->n_heads_kv);
  if (d->head_dim == 128)
    return d->format == LOOPVQ_MX_E4M3 ? attn_variant_t<128, LOOPVQ_MX_E4M3>(rows, fine)
                                       : attn_variant_t<128, LOOPVQ_MX_E2M1>(rows, fine);
  return d->format == LOOPVQ_MX_E4M3 ? attn_variant_t<64, LOOPVQ_MX_E4M3>(rows, fine)
                                     : attn_variant_t<64, LOOPVQ_MX_E2M1>(rows, fine);
}
// Blocks of the launch: no more than there are warps' worth of tiles.
int attn_grid(const loopvq_mx_desc* d, const loopvq_mx_layout* l, const AttnVariant& v) {
  const int64_t rows = (int64_t)l->max_new * (d->n_heads_q / d->n_heads_kv);
  const int64_t chunks = (rows + v.chunk - 1) / v.chunk, tiles = ((int64_t)l->max_ctx_len + kMxTile - 1) / kMxTile;
  const int most = v.workers / v.per_block;
  const int64_t each = (int64_t)d->n_heads_kv * chunks * tiles;   // below 2^62
  if (each >= v.workers) return most;
  const int64_t n = (each * l->batch + v.per_block - 1) / v.per_block;
  return n < 1 ? 1 : n < most ? (int)n : most;
}

// How many parts a unit has is known on the device only; with full lengths it is
// workers / units.  From 24 on a block per row (8 rows of 16 heads over 32K, 100
// parts: 45.5 us in all against 59), below that a warp per row.
template <int D, int CHUNK>
loopvq_status launch_merge(const MxAttnParams& p, int64_t rows, cudaStream_t s) {
  const int64_t units = (int64_t)p.L.batch * p.H * ((rows + CHUNK - 1) / CHUNK);
  const bool many_parts = p.n_workers > 24 * units;
  const int most = (int)(rows < CHUNK ? rows : CHUNK);
  const cudaError_t e =
      many_parts ? mx_launch(mx_merge_kernel<D, CHUNK>, dim3((p.n_workers + kMergeHeads - 1) / kMergeHeads, most < 16 ? most : 16),
                             kMergeWarps * 32, 0, s, p)
                 : mx_launch(mx_merge_rows_kernel<D, CHUNK>, dim3(p.n_workers, (most + kMergeWarps - 1) / kMergeWarps),
                             kMergeWarps * 32, 0, s, p);
  return e == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}
template <int D, int FMT, int NARROW, int TERMS, int NT>
loopvq_status launch_attn(const MxAttnParams& p, int grid, int64_t rows, cudaStream_t s) {
  constexpr int smem = MxRing<D, FMT, NARROW, NT>::kBytes, W = MxRing<D, FMT, NARROW, NT>::kWarps, CHUNK = MxRows<D, NARROW>::kPerGroup * NT;
  auto kfn = TERMS == 2 || p.softcap > kFastCap ? mx_attn_kernel<D, FMT, NARROW, TERMS, NT, true>
                                                : mx_attn_kernel<D, FMT, NARROW, TERMS, NT, TERMS == 2>;
  if (cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return LOOPVQ_ERR_CUDA;
  if (mx_launch(kfn, dim3(grid), (W + 1) * 32, smem, s, p) != cudaSuccess) return LOOPVQ_ERR_CUDA;
  return launch_merge<D, CHUNK>(p, rows, s);
}
template <int D, int FMT>
loopvq_status launch_attn_v(const MxAttnParams& p, const AttnVariant& v, bool fine, int grid, int64_t rows,
                            cudaStream_t s) {
  if (v.rows)
    return mx_rows_launch(D, FMT, p, grid, s) == cudaSuccess ? launch_merge<D, kMxRowsChunk>(p, rows, s) : LOOPVQ_ERR_CUDA;
  if (v.narrow == 2) return fine ? launch_attn<D, FMT, 2, 2, 1>(p, grid, rows, s) : launch_attn<D, FMT, 2, 1, 1>(p, grid, rows, s);
  if (v.narrow)
    return fine ? launch_attn<D, FMT, 1, 2, 1>(p, grid, rows, s)
                : v.nt == 2 ? launch_attn<D, FMT, 1, 1, 2>(p, grid, rows, s) : launch_attn<D, FMT, 1, 1, 1>(p, grid, rows, s);
  if (fine) return v.nt == 2 ? launch_attn<D, FMT, 0, 2, 2>(p, grid, rows, s) : launch_attn<D, FMT, 0, 2, 1>(p, grid, rows, s);
  return v.nt == 2 ? launch_attn<D, FMT, 0, 1, 2>(p, grid, rows, s) : launch_attn<D, FMT, 0, 1, 1>(p, grid, rows, s);
}

loopvq_status attn_checks(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout, MxLayout* L) {
  loopvq_status st = mx_check_desc(desc);
  if (st != LOOPVQ_OK) return st;
  st = mx_check_layout(layout, L);
  if (st != LOOPVQ_OK) return st;
  return layout->max_new > kMxMaxTree ? LOOPVQ_ERR_UNSUPPORTED : LOOPVQ_OK;
}
struct AttnWs {
  size_t partials_off, total;
};
AttnWs attn_ws(const loopvq_mx_desc* desc, int grid, const AttnVariant& v) {
  const size_t warps = (size_t)grid * v.per_block;
  AttnWs w;
  w.partials_off = (warps * sizeof(int4) + 255) & ~(size_t)255;
  w.total = w.partials_off + warps * 2 * v.chunk * (desc->head_dim + 4) * sizeof(float);
  return w;
}

}  // namespace
}  // namespace loopvq

using namespace loopvq;

extern "C" size_t loopvq_mx_attn_workspace_bytes(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout) {
  MxLayout L;
  if (attn_checks(desc, layout, &L) != LOOPVQ_OK) return 0;
  size_t most = 0;   // of both precisions
  for (int fine = 0; fine < 2; ++fine) {
    const AttnVariant v = attn_variant(desc, layout, fine);
    const size_t n = attn_ws(desc, attn_grid(desc, layout, v), v).total;
    if (n > most) most = n;
  }
  return most;
}

extern "C" loopvq_status loopvq_mx_attn(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout,
                                        const void* poolK, const void* poolV, const void* q, loopvq_dtype q_dtype,
                                        int64_t q_stride_n, int64_t q_stride_h, const uint64_t* tree_mask,
                                        int32_t loop_step, float softmax_scale, float softcap, const float* slopes,
                                        void* out, loopvq_dtype out_dtype, float* lse_out, void* workspace,
                                        size_t workspace_bytes, uint32_t* fault_bits, loopvq_stream_t stream) {
  MxAttnParams p = {};
  const loopvq_status st = attn_checks(desc, layout, &p.L);
  if (st != LOOPVQ_OK) return st;
  if (mx_pool_bytes(desc, layout->pool_tokens) == 0) return LOOPVQ_ERR_UNSUPPORTED;
  if (loop_step < 0 || loop_step >= desc->n_loop) return LOOPVQ_ERR_INVALID_ARG;
  if (!poolK || !poolV || ((uintptr_t)poolK & 15) || ((uintptr_t)poolV & 15)) return LOOPVQ_ERR_INVALID_ARG;
  if ((q_dtype != LOOPVQ_F32 && q_dtype != LOOPVQ_BF16) || (out_dtype != LOOPVQ_F32 && out_dtype != LOOPVQ_BF16))
    return LOOPVQ_ERR_INVALID_ARG;
  if (q_stride_n < 0 || q_stride_h < 0 || !(softcap >= 0.f) || !(softcap <= 3.0e38f) ||
      !(softmax_scale >= -3.0e38f && softmax_scale <= 3.0e38f))
    return LOOPVQ_ERR_INVALID_ARG;
  if (((uintptr_t)tree_mask & 7) || ((uintptr_t)slopes & 3) || ((uintptr_t)lse_out & 3) || ((uintptr_t)fault_bits & 3))
    return LOOPVQ_ERR_INVALID_ARG;
  if (layout->total_new == 0 || layout->max_new == 0 || layout->max_ctx_len == 0) return LOOPVQ_OK;
  const uintptr_t qs = q_dtype == LOOPVQ_BF16 ? 2 : 4;
  if (!q || (uintptr_t)q % qs || !out || ((uintptr_t)out & 15)) return LOOPVQ_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255)) return LOOPVQ_ERR_INVALID_ARG;
  // two fp16 terms of q and of the weights
  const bool fine = q_dtype == LOOPVQ_F32 || out_dtype == LOOPVQ_F32;
  const AttnVariant v = attn_variant(desc, layout, fine);
  const int grid = attn_grid(desc, layout, v);
  const AttnWs ws = attn_ws(desc, grid, v);
  if (workspace_bytes < ws.total) return LOOPVQ_ERR_WORKSPACE_TOO_SMALL;
  const size_t step = (size_t)desc->n_heads_kv * p.L.pool_tiles * mx_tile_bytes(desc->head_dim, desc->format);
  p.H = desc->n_heads_kv;
  p.Hq = desc->n_heads_q;
  p.G = p.Hq / p.H;
  p.pk = (const uint8_t*)poolK + loop_step * step;
  p.pv = (const uint8_t*)poolV + loop_step * step;
  p.q = q;
  p.q_bf16 = q_dtype == LOOPVQ_BF16;
  p.q_vec = !(((uintptr_t)q | (uintptr_t)q_stride_n * qs | (uintptr_t)q_stride_h * qs) & 15);
  p.qn = q_stride_n;
  p.qh = q_stride_h;
  p.tree_mask = tree_mask;
  p.softcap = softcap;
  p.scale = softmax_scale * (softcap > 0.f ? 0.25f : 0.25f * kLog2e);
  p.inv_cap = softcap > 0.f ? std::fmin(1.f / softcap, 0x1p126f) : 0.f;   // of a smaller cap every score but 0 is at it
  p.inv_cap2 = 2.f * kLog2e * p.inv_cap;
  p.slopes = slopes;
  p.out = out;
  p.out_bf16 = out_dtype == LOOPVQ_BF16;
  p.lse = lse_out;
  p.n_workers = grid * v.per_block;
  p.headers = (int4*)workspace;
  p.partials = (float*)((uint8_t*)workspace + ws.partials_off);
  p.fault = fault_bits;
  const int64_t rows = (int64_t)layout->max_new * p.G;
  cudaStream_t s = (cudaStream_t)stream;
  if (desc->head_dim == 128)
    return desc->format == LOOPVQ_MX_E4M3 ? launch_attn_v<128, LOOPVQ_MX_E4M3>(p, v, fine, grid, rows, s)
                                          : launch_attn_v<128, LOOPVQ_MX_E2M1>(p, v, fine, grid, rows, s);
  return desc->format == LOOPVQ_MX_E4M3 ? launch_attn_v<64, LOOPVQ_MX_E4M3>(p, v, fine, grid, rows, s)
                                        : launch_attn_v<64, LOOPVQ_MX_E2M1>(p, v, fine, grid, rows, s);
}
