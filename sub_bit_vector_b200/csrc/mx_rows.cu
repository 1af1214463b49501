// Attention over the microscaled KV cache for requests with many query rows
// (trees of drafts, several query heads per KV head), on the tcgen05 tensor
// cores.  bf16 queries and outputs.
//
// A block takes a share of the list of tiles as a warp of mx_attn_kernel does;
// a chunk is 128 rows = the 128 lanes of the accumulators, one thread per row,
// so that a row's softmax needs no exchange.  Per tile of 32 tokens:
//   K' (fp16, shared memory) = code * 2^(e - E), E the token's largest scale
//     exponent; S[128 x 32] = Q K'^T (Q and S in TMEM), x = S 2^E * scale in fp32.
//   P (fp16, TMEM) = 2^(x + E - M), E the largest exponent of the token's value,
//     M a reference per row, raised as in mx_attn.cu; V' = code * 2^(e - E);
//     O[128 x D] += P V'.
// K' and V' are exact as long as a code times 2^(e - E) is an fp16 number; below,
// an element is rounded to 2^-24 of 2^E, which is less than 2^-26 of its token's
// largest element.  A block of NaN counts as 0 in V' and is put into the outputs
// of the rows that see it at the end.
// Four warps convert codes, one of which issues the scores' product; four
// compute the softmax, one of which issues P V and another the copies.  Operands
// and scores are double-buffered, so that tile i's softmax, tile i + 1's scores
// and the product P V of tile i - 1 run together.
//
// P is one fp16 term, as in mx_attn.cu and for its reason.
//
// A tree of 64 nodes, two query heads per KV head, over 32K tokens of 16 heads x
// 128, e2m1: 115 us (the warps' kernel 253).  34 GFLOP would take 21 us.  Issue slots
// are 47% and the tensor pipe 14% busy: the 16 warps of an SM (128 registers each,
// 264 bytes of a row's query spilled at D = 128, 44 at 64) mostly wait for one another, at
// a block barrier and five mbarriers per 32 tokens.
//
// Operands in shared memory are K-major without swizzle: core matrices of 8
// rows x 16 bytes, at (row / 8) * SBO + (k / 8) * LBO.  LBO and SBO are padded so
// that the lanes of a store, in the order in which they hold codes, hit
// different banks.
#include "mx_attn.cuh"

namespace loopvq {
namespace {

constexpr int kRowsThreads = 2 * kMxRowsChunk;   // softmax, conversion

template <int D, int FMT>
struct Rows {
  using Tile = MxTile<D, FMT>;
  static constexpr int NB = Tile::kBlocks;
  static constexpr int kStages = 4;
  static constexpr int kKLbo = 160, kKSbo = D / 8 * 160;                 // tokens x channels
  static constexpr int kVLbo = 144, kVSbo = 672, kVBlock = 4 * kVSbo;    // channels x tokens, per block
  static constexpr int kKBuf = kMxTile / 8 * kKSbo, kVBuf = NB * kVBlock;
  static constexpr int kK = 0, kV = kK + 2 * kKBuf, kRing = kV + 2 * kVBuf,
                       kSlot = 2 * Tile::kBytes, kInfo = kRing + kStages * kSlot;
  static constexpr int kNeed = kInfo + 1024;
  static constexpr int kBytes = kNeed > 76 * 1024 ? kNeed : 76 * 1024;   // two blocks per SM, no third that would wait for TMEM
  // TMEM columns: O, Q (two fp16 per column), and twice S, over which P is written
  static constexpr int kO = 0, kQ = D, kS = D + D / 2, kCols = 256;
  static_assert(kS + 2 * kMxTile <= kCols, "TMEM");
};
// What the converting warps tell the others: per tile in turn, and barriers.
struct RowsInfo {
  struct alignas(16) {
    float fac[kMxTile];    // 2^E of each key
    float vfac[kMxTile];   // of each value, NaN left out
    int pos[kMxTile];      // positions (with slopes)
    uint8_t nan[4][4];     // [block][quarter]: tokens whose value is NaN there
    float vmax[4];         // largest of vfac in each quarter
    uint32_t hidden;       // the page is not in the pool
  } t[2];
  uint64_t full[4], freed[4];                     // raw tiles: arrived, read
  uint64_t told[2], ready[2], scores[2], weights[2], sums[2];   // info, V' written; S, P, O += P V done
  uint64_t query;                                 // Q written
  uint32_t tmem, bad;
};

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 | (uint64_t)((sbo >> 4) & 0x3FFF) << 32 |
         (uint64_t)1 << 46;   // descriptor version; no swizzle
}
// kind::f16, fp16 operands, K-major, fp32 sums, M = 128
constexpr uint32_t idesc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kMxRowsChunk >> 4) << 24);
}
// Issued by a whole warp with the same arguments, of which the elected thread
// acts: the arguments then stay in uniform registers, without which the eight
// instructions of a score tile took 1000 cycles to issue.
__device__ __forceinline__ uint32_t elect() {
  uint32_t e;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
  return e;
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc, uint32_t e) {   // A in TMEM
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(e)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar, uint32_t e) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(e)
      : "memory");
}
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
// 32 columns of this warp's lanes, waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t mul_f16(uint32_t a, uint32_t s) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(s));
  return r;
}
// 2^(e - E) as fp32 from 2^e and 2^E, 0 where it would be below 2^-126.
__device__ __forceinline__ float ratio(float e, float E) {
  return __int_as_float(max(__float_as_int(e) - __float_as_int(E) + 0x3f800000, 0));
}

template <int D, int FMT, bool EXACT>
__global__ void __launch_bounds__(kRowsThreads, 2) mx_rows_kernel(const MxAttnParams p) {
  using R = Rows<D, FMT>;
  using Tile = MxTile<D, FMT>;
  constexpr int NB = R::NB, S = R::kStages, CHUNK = kMxRowsChunk;
  extern __shared__ __align__(1024) uint8_t sm[];
  static_assert(sizeof(RowsInfo) <= 1024 && S <= 4, "");
  RowsInfo& I = *reinterpret_cast<RowsInfo*>(sm + R::kInfo);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  mx_begin();

  // this block's share of the list of tiles
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
  const int wid = blockIdx.x;
  const int64_t share = total / p.n_workers;
  const int extra = (int)(total % p.n_workers);
  const int64_t begin = wid * share + min(wid, extra);
  const int count = (int)share + (wid < extra);
  if (threadIdx.x == 0) p.headers[wid] = make_int4(0, 0, 0, 0);
  if (count == 0) return;   // the whole block
  MxCursor cc = mx_seek<CHUNK>(p, begin, u0, t0, lane);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&I.tmem)), "r"(R::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 160) {
    for (int i = 0; i < S; ++i) {
      mbar_init(smem_u32(&I.full[i]), 1);
      mbar_init(smem_u32(&I.freed[i]), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&I.told[i]), 4);
      mbar_init(smem_u32(&I.ready[i]), 4);
      mbar_init(smem_u32(&I.scores[i]), 1);
      mbar_init(smem_u32(&I.weights[i]), 128);
      mbar_init(smem_u32(&I.sums[i]), 1);
    }
    mbar_init(smem_u32(&I.query), 128);
    I.bad = 0;
    fence_mbar_init();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = I.tmem;
  // Use n of a barrier that alternates between two: its parity.
  auto wait2 = [&](uint64_t* bars, int n) { return mbar_wait_bounded(smem_u32(bars + (n & 1)), (uint32_t)(n >> 1) & 1); };
  bool ok = true;   // no wait has run out
  int done = 0;     // tiles

  if (warp >= 4) {
    // ======================== conversion, copies, products
    const int w4 = __shfl_sync(0xffffffffu, warp - 4, 0);
    const bool leader = w4 == 0;   // issues S
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t desc_k = smem_desc(smem_u32(sm + R::kK), R::kKLbo, R::kKSbo);
    const int sub = w4 >> 1;
    constexpr int UB = NB / 2;   // blocks of a warp, of one half of the tile
    const int b0 = (w4 & 1) * UB;
    int slot = 0;
    uint32_t phase = 0;
    // Barrier of these warps; false, in all threads alike, once a wait has run out in any.
    auto sync4 = [&]() {
      uint32_t failed;
      asm volatile(
          "{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n bar.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
          : "=r"(failed)
          : "r"(ok ? 0u : 1u)
          : "memory");
      return ok = failed == 0;
    };
    bool go = true;
    int units = 0;
    while (done < count && go) {
      MxReq rq = {};
      mx_request(p.L, cc.r, &rq, nullptr);
      const int first_tile = cc.t, n_tiles = min(cc.tiles - cc.t, count - done);
      const uint64_t all_new = rq.n >= 64 ? ~0ull : (1ull << rq.n) - 1;
      for (int it = 0; it < n_tiles; ++it) {
        const int i = done;
        auto& T = I.t[i & 1];
        const int tok0 = (first_tile + it) * kMxTile;
        const bool edge = tok0 + kMxTile > rq.base;
        ok &= mbar_wait_bounded(smem_u32(&I.full[slot]), phase);
        const bool bad = *reinterpret_cast<volatile uint32_t*>(&I.bad) >> slot & 1;
        if (i >= 2) ok &= wait2(I.weights, i - 2);   // K' and the info of tile i - 2 have been read
        const uint8_t* const sk = sm + R::kRing + slot * R::kSlot;
        const uint8_t* const sv = sk + Tile::kBytes;
        uint32_t w[UB][4], wv[UB][4];   // e4m3: 4 words of a block; e2m1: 2
        auto load_codes = [&](const uint8_t* tile, uint32_t (&w)[UB][4]) {
#pragma unroll
          for (int k = 0; k < UB; ++k) {
            if constexpr (FMT == LOOPVQ_MX_E4M3) {
              const uint4 z = *reinterpret_cast<const uint4*>(tile + mx_code_off<D, FMT>(sub, b0 + k, lane));
              w[k][0] = z.x; w[k][1] = z.y; w[k][2] = z.z; w[k][3] = z.w;
            } else {
              const uint2 z = *reinterpret_cast<const uint2*>(tile + mx_code_off<D, FMT>(sub, b0 + k, lane));
              w[k][0] = z.x; w[k][1] = z.y; w[k][2] = w[k][3] = 0;
            }
            if (bad) w[k][0] = w[k][1] = w[k][2] = w[k][3] = 0;
          }
        };
        // ---- K'
        load_codes(sk, w);
        load_codes(sv, wv);
        uint32_t scw[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) scw[b] = *reinterpret_cast<const uint32_t*>(sk + mx_scale_off<D, FMT>(sub * 4 + (g >> 1), b));
        uint8_t* const dk = sm + R::kK + (i & 1) * R::kKBuf;
#pragma unroll
        for (int ab = 0; ab < 2; ++ab) {
          const int sh = 8 * ((g & 1) + 2 * ab), n = sub * 16 + 4 * (g >> 1) + (g & 1) + 2 * ab;
          float ke[NB], top = 0.f;   // 255: infinity, which turns the score into NaN
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            ke[b] = __uint_as_float((scw[b] >> sh & 255u) << 23);
            top = fmaxf(top, ke[b]);
          }
          if ((w4 & 1) == 0 && c == 0) T.fac[n] = top;
#pragma unroll
          for (int k = 0; k < UB; ++k) {
            uint32_t hc[4];
            if constexpr (FMT == LOOPVQ_MX_E4M3) {
              codes_e4m3(w[k][2 * ab], hc);
              codes_e4m3(w[k][2 * ab + 1], hc + 2);
            } else {
              codes_e2m1(w[k][ab], hc);
            }
            const float own = ratio(b0 ? ke[NB - UB + k] : ke[k], top);
            const uint32_t s2 = pack_f16(own, own);
            *reinterpret_cast<uint4*>(dk + (n >> 3) * R::kKSbo + (4 * (b0 + k) + c) * R::kKLbo + (n & 7) * 16) =
                make_uint4(mul_f16(hc[0], s2), mul_f16(hc[1], s2), mul_f16(hc[2], s2), mul_f16(hc[3], s2));
          }
        }
        {   // V's factors: a warp has 8 tokens, a lane a block of one
          const int vt = lane / NB & 7, vb = lane % NB;
          const uint32_t ve = sv[mx_scale_off<D, FMT>(2 * w4 + (vt >> 2), vb) + (vt & 3)];
          const bool is_nan = ve == kMxNan;
          float top = is_nan ? 0.f : __uint_as_float(ve << 23);
#pragma unroll
          for (int d = 1; d < NB; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // not negative
          const uint32_t nans = __ballot_sync(0xffffffffu, is_nan);
          if (vb == 0) T.vfac[8 * w4 + vt] = top;
          if (lane < NB) {
            uint32_t z = 0;
            if (nans) {
              for (int t = 0; t < 8; ++t) z |= (nans >> (t * NB + lane) & 1u) << t;
            }
            T.nan[lane][w4] = (uint8_t)z;
          }
          if (lane == 0) {
            T.vmax[w4] = __uint_as_float(most);
            if (w4 == 0) T.hidden = bad;
          }
        }
        if (p.slopes && w4 == 0) {
          const int j = tok0 + lane - rq.base;
          int at = tok0 + lane;
          if (j >= 0 && j < rq.n) {
            const uint64_t its = p.tree_mask ? ld_once(p.tree_mask + rq.row0 + j) & all_new : (2ull << j) - 1;
            at = rq.base + __popcll(its & ~(1ull << j));
          }
          T.pos[lane] = at;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&I.told[i & 1]));
        fence_proxy_async();
        if (!(go = sync4())) break;
        if (leader) {
          if (it == 0) ok &= mbar_wait_bounded(smem_u32(&I.query), (uint32_t)units & 1);
          if (i >= 2) ok &= wait2(I.sums, i - 2);   // P of tile i - 2, where S goes, has been read
          __syncwarp();
          tmem_after();
          const uint32_t el = elect();
          const uint64_t d = desc_k + (uint64_t)(i & 1) * (R::kKBuf >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_ts(tm + R::kS + (i & 1) * kMxTile, tm + R::kQ + 8 * k, d + k * (2 * R::kKLbo >> 4), idesc(kMxTile), k > 0, el);
          umma_commit(smem_u32(&I.scores[i & 1]), el);
        }
        // ---- V'
        const float4 ve = *reinterpret_cast<const float4*>(T.vfac + sub * 16 + 4 * c);   // of this lane's tokens
        if (i >= 2) ok &= wait2(I.sums, i - 2);   // V' of tile i - 2 has been read
        uint8_t* const dv = sm + R::kV + (i & 1) * R::kVBuf;
#pragma unroll
        for (int k = 0; k < UB; ++k) {
          uint32_t hv[4][2];   // [channel j][token pair]
          if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
            for (int j = 0; j < 4; ++j) codes_e4m3(edge ? drop_nan_codes(wv[k][j]) : wv[k][j], hv[j]);
          } else {
            codes_e2m1(wv[k][0], hv[0]);
            codes_e2m1(wv[k][1], hv[2]);
          }
          // a NaN block's ratio is large: its codes are 0, and so is what it gives
          const uint32_t z = *reinterpret_cast<const uint32_t*>(sv + mx_scale_off<D, FMT>(sub * 4 + c, b0 + k));
          const uint32_t s01 = pack_f16(fminf(ratio(scale_f32(z, 0), ve.x), 1.f), fminf(ratio(scale_f32(z, 1), ve.y), 1.f));
          const uint32_t s23 = pack_f16(fminf(ratio(scale_f32(z, 2), ve.z), 1.f), fminf(ratio(scale_f32(z, 3), ve.w), 1.f));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 4 * g + j;
            *reinterpret_cast<uint2*>(dv + (b0 + k) * R::kVBlock + (r >> 3) * R::kVSbo + (2 * sub + (c >> 1)) * R::kVLbo +
                                      (r & 7) * 16 + (c & 1) * 8) =
                make_uint2(mul_f16(hv[j][0], s01), mul_f16(hv[j][1], s23));
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&I.ready[i & 1]));
          mbar_arrive(smem_u32(&I.freed[slot]));
        }
        if (++slot == S) {
          slot = 0;
          phase ^= 1;
        }
        ++done;
      }
      ++units;
      if (done < count && go) mx_next_unit<CHUNK>(p, &cc);
    }
    if (!ok && lane == 0) set_fault(p.fault, LOOPVQ_FAULT_TIMEOUT);
  } else {
    // ======================== softmax: a thread has a row
    const int tid = threadIdx.x;
    const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);   // this warp's lanes
    const bool adder = __shfl_sync(0xffffffffu, warp, 0) == 0;    // issues P V
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t desc_v = smem_desc(smem_u32(sm + R::kV), R::kVLbo, R::kVSbo);
    MxCursor pc = cc;            // the copier's: the next tile
    const int per = p.L.page_tokens / kMxTile;
    int page = pc.t / per, in_page = pc.t % per, issued = 0;
    int64_t head = 0;
    int id = 0;
    auto issue = [&](int slot) {   // by the copier
      const uint32_t bar = smem_u32(&I.full[slot]), dst = smem_u32(sm + R::kRing + slot * R::kSlot);
      if (id >= 0 && id < p.L.n_pages) {
        const int64_t at = (head + (int64_t)id * per + in_page) * Tile::kBytes;
        mbar_arrive_expect_tx(bar, 2 * Tile::kBytes);
        bulk_g2s(dst, p.pk + at, Tile::kBytes, bar);
        bulk_g2s(dst + Tile::kBytes, p.pv + at, Tile::kBytes, bar);
      } else {
        set_fault(p.fault, LOOPVQ_FAULT_POOL_RANGE);
        atomicOr(&I.bad, 1u << slot);   // before the arrival that publishes it
        mbar_arrive(bar);
      }
      if (++issued < count) {
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
    };
    const bool copier = tid == 96;
    if (copier) {
      head = (int64_t)(pc.u / (pc.units / p.H)) * p.L.pool_tiles;
      id = ld_once(p.L.pages + (int64_t)pc.r * p.L.max_pages + page);
      for (int i = 0; i < S && i < count; ++i) issue(i);
    }
    int slot = 0;
    uint32_t phase = 0;
    while (done < count && ok) {
      MxReq rq = {};
      mx_request(p.L, cc.r, &rq, nullptr);
      const int chunks = cc.units / p.H, h = cc.u / chunks, rho0 = (cc.u - h * chunks) * CHUNK;
      const int rows = max(0, min(CHUNK, rq.n * p.G - rho0));   // 0 if lengths change meanwhile
      const int first_tile = cc.t, n_tiles = min(cc.tiles - cc.t, count - done);
      const uint64_t all_new = rq.n >= 64 ? ~0ull : (1ull << rq.n) - 1;
      // the row: scaled by a power of two to a largest magnitude in [2^14, 2^15),
      // as fp16 (exact for bf16 down to 2^-28 of it).  The last unit's scores are
      // done: nothing reads Q any more.
      const int rho = rho0 + tid;
      const bool there = tid < rows;
      float f, slope = 0.f;
      uint64_t sees = 0;
      int pos_q = 0;
      {
        const int node = rho / p.G, hq = h * p.G + rho % p.G;
        const __nv_bfloat16* x =
            reinterpret_cast<const __nv_bfloat16*>(p.q) + (int64_t)(rq.row0 + node) * p.qn + (int64_t)hq * p.qh;
        float mx = 0.f;
        uint32_t q[D / 2];
#pragma unroll
        for (int k = 0; k < D / 2; ++k) q[k] = 0u;
        if (there) {
          if (p.q_vec) {
#pragma unroll
            for (int k = 0; k < D / 8; ++k) {
              const uint4 z = ld_once(reinterpret_cast<const uint4*>(x) + k);
              q[4 * k] = z.x; q[4 * k + 1] = z.y; q[4 * k + 2] = z.z; q[4 * k + 3] = z.w;
            }
          } else {
            const uint16_t* x16 = reinterpret_cast<const uint16_t*>(x);
#pragma unroll
            for (int k = 0; k < D / 2; ++k) q[k] = (uint32_t)x16[2 * k] | (uint32_t)x16[2 * k + 1] << 16;
          }
          sees = (p.tree_mask ? ld_once(p.tree_mask + rq.row0 + node) : (2ull << node) - 1) & all_new;
          pos_q = rq.base + __popcll(sees & ~(1ull << node));
          if (p.slopes) slope = ld_once(p.slopes + hq) * kLog2e;
        }
#pragma unroll
        for (int k = 0; k < D / 2; ++k) mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(q[k])), fabsf(bf16_hi(q[k]))));
        const int ex = max((int)(__float_as_uint(mx) >> 23), 1) - 127;
        const int k2 = min(14 - ex, 120);
        const float up = __uint_as_float((uint32_t)(127 + k2) << 23), down = __uint_as_float((uint32_t)(129 - k2) << 23);
        f = p.scale * down;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = pack_f16(bf16_lo(q[16 * k + j]) * up, bf16_hi(q[16 * k + j]) * up);
          __syncwarp();
          tmem_st16(mine + R::kQ + 16 * k, z);
        }
      }
      tmem_wait_st();
      tmem_before();
      mbar_arrive(smem_u32(&I.query));

      float m = -INFINITY, l = 0.f, M = -INFINITY, rs = 0.f;
      uint32_t poison = 0;   // bit b: the row sees a NaN of block b
      for (int it = 0; it < n_tiles; ++it) {
        const int i = done + it;
        const auto& T = I.t[i & 1];
        const int tok0 = (first_tile + it) * kMxTile;
        ok &= wait2(I.told, i);
        ok &= wait2(I.scores, i);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tmem_after();
        const bool hidden = T.hidden != 0, edge = hidden || tok0 + kMxTile > rq.base;
        float x[32];
        tmem_ld32(mine + R::kS + (i & 1) * kMxTile, x);
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int t = 0; t < 32; t += 4) {
          const float4 fc = *reinterpret_cast<const float4*>(T.fac + t);
          const float2 a = mul2(mul2(make_float2(x[t], x[t + 1]), f2), make_float2(fc.x, fc.y));
          const float2 b = mul2(mul2(make_float2(x[t + 2], x[t + 3]), f2), make_float2(fc.z, fc.w));
          x[t] = a.x;
          x[t + 1] = a.y;
          x[t + 2] = b.x;
          x[t + 3] = b.y;
        }
        if (p.softcap > 0.f) {
#pragma unroll
          for (int t = 0; t < 32; ++t)
            x[t] = EXACT ? capped(x[t], p.softcap, p.inv_cap) : capped_fast(x[t], p.softcap, p.inv_cap2);
        }
        if (p.slopes) {
#pragma unroll
          for (int t = 0; t < 32; ++t) x[t] -= slope * (float)(pos_q - T.pos[t]);
        }
        uint32_t vis = ~0u;   // bits of the tokens that the row sees
        if (edge) {
          const int lo = rq.base - tok0;   // the prefix's part of the tile
          vis = hidden ? 0u
                : lo >= 32 ? ~0u
                : lo > 0   ? ((1u << lo) - 1) | (uint32_t)(sees << lo)
                           : (uint32_t)(lo > -64 ? sees >> -lo : 0ull);
#pragma unroll
          for (int t = 0; t < 32; ++t)
            if (!(vis >> t & 1)) x[t] = -INFINITY;
        }
        if constexpr (NB == 4) {
          const uint4 z = *reinterpret_cast<const uint4*>(T.nan);
          poison |= (z.x & vis ? 1u : 0u) | (z.y & vis ? 2u : 0u) | (z.z & vis ? 4u : 0u) | (z.w & vis ? 8u : 0u);
        } else {
          const uint2 z = *reinterpret_cast<const uint2*>(T.nan);
          poison |= (z.x & vis ? 1u : 0u) | (z.y & vis ? 2u : 0u);
        }
        float tops[4] = {x[0], x[1], x[2], x[3]};   // four chains
#pragma unroll
        for (int t = 4; t < 32; ++t) tops[t & 3] = fmaxf(tops[t & 3], x[t]);
        const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        // ---- raise the references if a score or a weight could leave its range
        const bool over = top > m + kScoreSlack || ex2(top - (m == -INFINITY ? 0.f : m)) * fmaxf(fmaxf(T.vmax[0], T.vmax[1]), fmaxf(T.vmax[2], T.vmax[3])) * rs > kWeightMax;
        if (__any_sync(0xffffffffu, over)) {   // (all lanes: the TMEM accesses are the warp's)
          const float mn = fmaxf(m, top);
          if (m != -INFINITY) l *= ex2(m - mn);
          m = mn;
          float bm = -INFINITY;
#pragma unroll
          for (int t = 0; t < 32; ++t) bm = fmaxf(bm, x[t] + (float)((__float_as_int(T.vfac[t]) >> 23) - 127));
          const float Mn = fmaxf(M, bm - kWeightExp);
          const float back = M == -INFINITY ? 0.f : ex2(M - Mn);
          M = Mn;
          rs = Mn == -INFINITY ? 0.f : ex2(mn - Mn);
          if (it > 0) {
            ok &= wait2(I.sums, i - 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tmem_after();
#pragma unroll 1
            for (int b = 0; b < NB * 2; ++b) {
              float o[16];
              tmem_ld16(mine + R::kO + 16 * b, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] *= back;
              uint32_t z[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(o[e]);
              tmem_st16(mine + R::kO + 16 * b, z);
            }
          }
        }
        // ---- weights
        const float mi = m == -INFINITY ? 0.f : m;
        const float2 r2 = make_float2(rs, rs), n2 = make_float2(-mi, -mi);
        float2 sum = make_float2(0.f, 0.f), sum2 = sum;
        uint32_t pw[16];
#pragma unroll
        for (int t = 0; t < 32; t += 4) {
          float2 y = add2(make_float2(x[t], x[t + 1]), n2), z = add2(make_float2(x[t + 2], x[t + 3]), n2);
          y = make_float2(ex2(y.x), ex2(y.y));
          z = make_float2(ex2(z.x), ex2(z.y));
          sum = add2(sum, y);
          sum2 = add2(sum2, z);
          const float4 sc = *reinterpret_cast<const float4*>(T.vfac + t);
          const float2 wy = mul2(mul2(y, make_float2(sc.x, sc.y)), r2), wz = mul2(mul2(z, make_float2(sc.z, sc.w)), r2);
          pw[t / 2] = pack_f16(wy.x, wy.y);
          pw[t / 2 + 1] = pack_f16(wz.x, wz.y);
        }
        l += (sum.x + sum.y) + (sum2.x + sum2.y);
        __syncwarp();
        tmem_st16(mine + R::kS + kMxTile * (i & 1), pw);   // S has been read; P of tile i - 2 was, before S was written
        tmem_wait_st();
        tmem_before();
        mbar_arrive(smem_u32(&I.weights[i & 1]));
        if (adder) {   // O += P V'
          ok &= wait2(I.ready, i);
          ok &= wait2(I.weights, i);
          __syncwarp();
          tmem_after();
          const uint32_t el = elect(), pa = tm + R::kS + kMxTile * (i & 1);
          const uint64_t dv = desc_v + (uint64_t)(i & 1) * (R::kVBuf >> 4);
          umma_ts(tm + R::kO, pa, dv, idesc(D), it > 0, el);
          umma_ts(tm + R::kO, pa + 8, dv + (2 * R::kVLbo >> 4), idesc(D), 1, el);
          umma_commit(smem_u32(&I.sums[i & 1]), el);
        }
        if (copier) {   // refill the ring where the conversion has read it
          ok &= mbar_wait_bounded(smem_u32(&I.freed[slot]), phase);
          if (*reinterpret_cast<volatile uint32_t*>(&I.bad) >> slot & 1) atomicAnd(&I.bad, ~(1u << slot));
          if (issued < count) issue(slot);
        }
        if (++slot == S) {
          slot = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      done += n_tiles;

      // ---------------------------------------------- the unit's rows, or this block's part of them
      ok &= wait2(I.sums, done - 1);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tmem_after();
      const bool whole = first_tile == 0 && n_tiles == cc.tiles;
      float* part = p.partials + ((size_t)(2 * wid + (first_tile == 0)) * CHUNK + tid) * (D + 4);
      const int64_t at = (int64_t)(rq.row0 + rho / p.G) * p.Hq + h * p.G + rho % p.G;
      if (there) {
        if (!whole) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
        else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll 1
      for (int b = 0; b < NB * 2; ++b) {
        float o[16];
        __syncwarp();
        tmem_ld16(mine + R::kO + 16 * b, o);
        // a row that saw only NaN has no M: its l is NaN
        const float fb = poison >> (b >> 1) & 1 ? NAN : M == -INFINITY ? l : ex2(M - m) * inv;
#pragma unroll
        for (int e = 0; e < 16; ++e) o[e] *= fb;
        if (there && !whole) {
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(part + 16 * b + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else if (there) {
          uint32_t z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            z[e] = *reinterpret_cast<const uint32_t*>(&v);
          }
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at * D + 16 * b);
          dst[0] = make_uint4(z[0], z[1], z[2], z[3]);
          dst[1] = make_uint4(z[4], z[5], z[6], z[7]);
        }
      }
      __syncwarp();
      if (first_tile == 0 && !whole && tid == 0) {
        // the blocks after this one that hold the unit's other tiles
        const int64_t last = begin + done - n_tiles + cc.tiles - 1, longer = (int64_t)extra * (share + 1);
        const int64_t owner = last < longer ? last / (share + 1) : extra + (last - longer) / share;
        p.headers[wid] = make_int4((int)(owner - wid), rq.row0, h, rho0 << 8 | rows);
      }
      tmem_before();   // the next unit's first weights, and with them its first product, come after this
      if (done < count) mx_next_unit<CHUNK>(p, &cc);
    }
    if (!ok && lane == 0) set_fault(p.fault, LOOPVQ_FAULT_TIMEOUT);
    if (copier && !ok)   // copies that are still on their way end before the block does
      for (int i = max(0, issued - S); i < issued; ++i) mbar_wait_bounded(smem_u32(&I.full[i % S]), (uint32_t)(i / S) & 1);
  }
  // products that were issued have ended: the sums of the last one are waited for above
  if (!ok) {
    for (int i = 0; i < 2; ++i) {
      mbar_wait_bounded(smem_u32(&I.scores[i]), 0);
      mbar_wait_bounded(smem_u32(&I.scores[i]), 1);
    }
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(R::kCols));
}

template <int D, int FMT>
cudaError_t launch(const MxAttnParams& p, int grid, cudaStream_t s) {
  constexpr int smem = Rows<D, FMT>::kBytes;
  auto kfn = p.softcap > kFastCap ? mx_rows_kernel<D, FMT, true> : mx_rows_kernel<D, FMT, false>;
  const cudaError_t e = cudaFuncSetAttribute(kfn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return mx_launch(kfn, dim3(grid), kRowsThreads, smem, s, p);
}

}  // namespace

int mx_rows_workers() { return 2 * device_sm_count(); }

cudaError_t mx_rows_launch(int head_dim, int format, const MxAttnParams& p, int grid, cudaStream_t s) {
  if (head_dim == 128)
    return format == LOOPVQ_MX_E4M3 ? launch<128, LOOPVQ_MX_E4M3>(p, grid, s) : launch<128, LOOPVQ_MX_E2M1>(p, grid, s);
  return format == LOOPVQ_MX_E4M3 ? launch<64, LOOPVQ_MX_E4M3>(p, grid, s) : launch<64, LOOPVQ_MX_E2M1>(p, grid, s);
}

}  // namespace loopvq
