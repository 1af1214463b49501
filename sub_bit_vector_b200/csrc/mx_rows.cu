// Attention over the microscaled KV cache for requests with many query rows
// (trees of drafts, several query heads per KV head), on the tcgen05 tensor
// cores.  bf16 queries and outputs.
//
// A block takes a share of the list of tiles as a warp of mx_attn_kernel does;
// a chunk is 128 rows = the 128 lanes of the accumulators, one thread per row,
// so that a row's softmax needs no exchange.  Per tile of 32 tokens:
//   K' (fp16, shared memory) = code * 2^(e - E), E the token's largest scale
//     exponent; S[128 x 32] = Q K'^T (TMEM), x = S 2^E * scale in fp32.
//   P (fp16, TMEM) = 2^(x + E - M), E the largest exponent of the token's value,
//     M a reference per row, raised as in mx_attn.cu; V' = code * 2^(e - E);
//     O[128 x D] += P V'.
// K' and V' are exact as long as a code times 2^(e - E) is an fp16 number; below,
// an element is rounded to 2^-24 of 2^E, which is less than 2^-26 of its token's
// largest element.  A block of NaN counts as 0 in V' and is put into the outputs
// of the rows that see it at the end.
// All threads convert K' while the previous tile's P V runs, and V while the
// scores are computed; two blocks per SM fill each other's waits.
//
// Operands in shared memory are K-major without swizzle: core matrices of 8
// rows x 16 bytes, at (row / 8) * SBO + (k / 8) * LBO.  LBO and SBO are padded so
// that the lanes of a store, in the order in which they hold codes, hit
// different banks.
#include "mx_attn.cuh"

namespace loopvq {
namespace {

constexpr int kRowsThreads = kMxRowsChunk;

template <int D, int FMT>
struct Rows {
  using Tile = MxTile<D, FMT>;
  static constexpr int NB = Tile::kBlocks;
  static constexpr int kStages = 3;
  static constexpr int kQLbo = 128, kQSbo = D / 8 * 128;                 // rows x channels
  static constexpr int kKLbo = 160, kKSbo = D / 8 * 160;                 // tokens x channels
  static constexpr int kVLbo = 144, kVSbo = 672, kVBlock = 4 * kVSbo;    // channels x tokens, per block
  static constexpr int kQ = 0, kK = kQ + kMxRowsChunk / 8 * kQSbo, kV = kK + kMxTile / 8 * kKSbo,
                       kRing = kV + NB * kVBlock, kSlot = 2 * Tile::kBytes, kFac = kRing + kStages * kSlot,
                       kVs = kFac + kMxTile * 4, kNan = kVs + kMxTile * 4, kVmax = kNan + 16, kPos = kVmax + 16, kBars = kPos + kMxTile * 4,
                       kNeed = kBars + (kStages + 2) * 8 + 16;
  static constexpr int kBytes = kNeed > 76 * 1024 ? kNeed : 76 * 1024;   // two blocks per SM, no third that would wait for TMEM
  // TMEM columns: O, S, P
  static constexpr int kO = 0, kS = D, kP = D + kMxTile, kCols = D == 128 ? 256 : 128;
  static_assert(kP + 16 <= kCols, "TMEM");
};

__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFF) | (uint64_t)((lbo >> 4) & 0x3FFF) << 16 | (uint64_t)((sbo >> 4) & 0x3FFF) << 32 |
         (uint64_t)1 << 46;   // descriptor version; no swizzle
}
// kind::f16, fp16 operands, K-major, fp32 sums, M = 128
constexpr uint32_t idesc(int n) {
  return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kMxRowsChunk >> 4) << 24);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {   // A in TMEM
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
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
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
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

template <int D, int FMT>
__global__ void __launch_bounds__(kRowsThreads, 2) mx_rows_kernel(const MxAttnParams p) {
  using R = Rows<D, FMT>;
  using Tile = MxTile<D, FMT>;
  constexpr int NB = R::NB, S = R::kStages, CHUNK = kMxRowsChunk;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* const full = reinterpret_cast<uint64_t*>(sm + R::kBars);
  uint64_t* const bar_s = full + S;   // scores done
  uint64_t* const bar_o = bar_s + 1;  // P V done
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(bar_o + 1);
  float* const fac = reinterpret_cast<float*>(sm + R::kFac);   // 2^E of each token
  float* const vfac = reinterpret_cast<float*>(sm + R::kVs);    // of V, NaN left out
  float* const vmax = reinterpret_cast<float*>(sm + R::kVmax);  // their largest
  uint32_t* const vnan = reinterpret_cast<uint32_t*>(sm + R::kNan);   // [block]: tokens of which it is NaN
  int* const pos_k = reinterpret_cast<int*>(sm + R::kPos);       // positions of the tile's tokens (with slopes)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

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
  if (tid == 0) p.headers[wid] = make_int4(0, 0, 0, 0);
  if (count == 0) return;   // the whole block
  MxCursor cc = mx_seek<CHUNK>(p, begin, u0, t0, lane);

  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(R::kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) {
    for (int i = 0; i < S + 2; ++i) mbar_init(smem_u32(full + i), 1);
    fence_mbar_init();
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t mine = tmem + ((uint32_t)(warp * 32) << 16);   // this warp's lanes

  MxCursor pc = cc;   // thread 0 feeds the ring; all threads keep its place
  const int per = p.L.page_tokens / kMxTile;
  int page = pc.t / per, in_page = pc.t % per, issued = 0;
  uint32_t bad = 0;   // bit per slot: its tile's page is not in the pool
  int64_t head = (int64_t)(pc.u / (pc.units / p.H)) * p.L.pool_tiles;
  int id = __ldg(p.L.pages + (int64_t)pc.r * p.L.max_pages + page);
  auto issue = [&](int slot) {
    const bool ok = id >= 0 && id < p.L.n_pages;
    bad = (bad & ~(1u << slot)) | (ok ? 0u : 1u << slot);
    if (tid == 0) {
      const uint32_t bar = smem_u32(full + slot), dst = smem_u32(sm + R::kRing + slot * R::kSlot);
      if (ok) {
        const int64_t at = (head + (int64_t)id * per + in_page) * Tile::kBytes;
        mbar_arrive_expect_tx(bar, 2 * Tile::kBytes);
        bulk_g2s(dst, p.pk + at, Tile::kBytes, bar);
        bulk_g2s(dst + Tile::kBytes, p.pv + at, Tile::kBytes, bar);
      } else {
        set_fault(p.fault, LOOPVQ_FAULT_POOL_RANGE);
        mbar_arrive(bar);
      }
    }
    if (++issued < count) {
      if (++pc.t == pc.tiles) {
        mx_next_unit<CHUNK>(p, &pc);
        page = in_page = 0;
        head = (int64_t)(pc.u / (pc.units / p.H)) * p.L.pool_tiles;
        id = __ldg(p.L.pages + (int64_t)pc.r * p.L.max_pages);
      } else if (++in_page == per) {
        in_page = 0;
        ++page;
        id = __ldg(p.L.pages + (int64_t)pc.r * p.L.max_pages + page);
      }
    }
  };
  for (int i = 0; i < S && i < count; ++i) issue(i);

  int done = 0, slot = 0;
  uint32_t phase = 0, phase_s = 0, phase_o = 0;
  bool busy_o = false;   // a P V is on its way
  bool busy_s = false;
  bool lost = false;
  while (done < count && !lost) {
    MxReq rq = {};
    mx_request(p.L, cc.r, &rq, nullptr);
    const int chunks = cc.units / p.H, h = cc.u / chunks, rho0 = (cc.u - h * chunks) * CHUNK;
    const int rows = min(CHUNK, rq.n * p.G - rho0);
    const int first_tile = cc.t, n_tiles = min(cc.tiles - cc.t, count - done);
    const uint64_t all_new = rq.n >= 64 ? ~0ull : (1ull << rq.n) - 1;

    // this thread's row: scaled by a power of two to a largest magnitude in
    // [2^14, 2^15), as fp16 (exact for bf16 down to 2^-28 of it)
    const int rho = rho0 + tid;
    const bool there = tid < rows;
    float f, slope = 0.f;
    uint64_t sees = 0;
    int pos_q = 0;
    {
      const int node = rho / p.G, hq = h * p.G + rho % p.G;
      float q[D];
      float mx = 0.f;
      if (there) {
        const int64_t at = (int64_t)(rq.row0 + node) * p.qn + (int64_t)hq * p.qh;
#pragma unroll
        for (int k = 0; k < D; k += 8) load_query<__nv_bfloat16>(p.q, at + k, p.q_vec, q + k);
        sees = (p.tree_mask ? __ldg(p.tree_mask + rq.row0 + node) : (2ull << node) - 1) & all_new;
        pos_q = rq.base + __popcll(sees & ~(1ull << node));
        if (p.slopes) slope = __ldg(p.slopes + hq) * kLog2e;
      } else {
#pragma unroll
        for (int k = 0; k < D; ++k) q[k] = 0.f;
      }
#pragma unroll
      for (int k = 0; k < D; ++k) mx = fmaxf(mx, fabsf(q[k]));
      const int ex = max((int)(__float_as_uint(mx) >> 23), 1) - 127;
      const int k2 = min(14 - ex, 120);
      const float up = __uint_as_float((uint32_t)(127 + k2) << 23), down = __uint_as_float((uint32_t)(127 - k2) << 23);
      f = p.softcap > 0.f ? p.scale / p.softcap * down : p.scale * kLog2e * down;
#pragma unroll
      for (int k = 0; k < D; k += 8)
        *reinterpret_cast<uint4*>(sm + R::kQ + (tid >> 3) * R::kQSbo + (k >> 3) * R::kQLbo + (tid & 7) * 16) =
            make_uint4(pack_f16(q[k] * up, q[k + 1] * up), pack_f16(q[k + 2] * up, q[k + 3] * up),
                       pack_f16(q[k + 4] * up, q[k + 5] * up), pack_f16(q[k + 6] * up, q[k + 7] * up));
    }
    float m = -INFINITY, l = 0.f, M = -INFINITY, rs = 0.f;
    uint32_t poison = 0;   // bit b: the row sees a NaN of block b
    bool first = true;   // no tile of the unit is in O yet

    for (int it = 0; it < n_tiles; ++it) {
      const int tok0 = (first_tile + it) * kMxTile;
      const bool edge = tok0 + kMxTile > rq.base;
      const bool skip = bad >> slot & 1;
      lost |= !mbar_wait_bounded(smem_u32(full + slot), phase);
      const uint8_t* const sk = sm + R::kRing + slot * R::kSlot;
      const uint8_t* const sv = sk + Tile::kBytes;
      if (!skip) {
        // ---- K', and the factors of scores and weights.  A warp converts half a tile of two blocks (D = 64: of one).
        const int sub = warp >> 1;
        constexpr int UB = NB / 2;   // blocks of a warp
        const int b0 = (warp & 1) * UB;
        uint32_t w[UB][4] = {};      // e4m3: 4 words of a block; e2m1: 2
        auto load_codes = [&](const uint8_t* tile) {
          if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
            for (int k = 0; k < UB; ++k) {
              const uint4 z = *reinterpret_cast<const uint4*>(tile + mx_code_off<D, FMT>(sub, b0 + k, lane));
              w[k][0] = z.x; w[k][1] = z.y; w[k][2] = z.z; w[k][3] = z.w;
            }
          } else {
#pragma unroll
            for (int k = 0; k < UB; ++k) {
              const uint2 z = *reinterpret_cast<const uint2*>(tile + mx_code_off<D, FMT>(sub, b0 + k, lane));
              w[k][0] = z.x; w[k][1] = z.y;
            }
          }
        };
        load_codes(sk);
        const int quad = sub * 4 + (g >> 1);
        uint32_t scw[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) scw[b] = *reinterpret_cast<const uint32_t*>(sk + mx_scale_off<D, FMT>(quad, b));
#pragma unroll
        for (int ab = 0; ab < 2; ++ab) {
          const int sh = 8 * ((g & 1) + 2 * ab), n = sub * 16 + 4 * (g >> 1) + (g & 1) + 2 * ab;
          float ke[NB], top = 0.f;   // 255: infinity, which turns the score into NaN
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            ke[b] = __uint_as_float((scw[b] >> sh & 255u) << 23);
            top = fmaxf(top, ke[b]);
          }
          if ((warp & 1) == 0 && c == 0) fac[n] = top;
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
            *reinterpret_cast<uint4*>(sm + R::kK + (n >> 3) * R::kKSbo + (4 * (b0 + k) + c) * R::kKLbo + (n & 7) * 16) =
                make_uint4(mul_f16(hc[0], s2), mul_f16(hc[1], s2), mul_f16(hc[2], s2), mul_f16(hc[3], s2));
          }
        }
        if (warp == 3 && lane < 8) {   // V's factors: a lane has a quad of tokens
          float top[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t nan[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t z = *reinterpret_cast<const uint32_t*>(sv + mx_scale_off<D, FMT>(lane, b));
            nan[b] = 0;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const float y = scale_f32(z, t);
              if (y == INFINITY) nan[b] |= 1u << (4 * lane + t);
              else top[t] = fmaxf(top[t], y);
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) nan[b] |= __shfl_xor_sync(0xffu, nan[b], d);
            if (lane == 0) vnan[b] = nan[b];
          }
          *reinterpret_cast<float4*>(vfac + 4 * lane) = make_float4(top[0], top[1], top[2], top[3]);
          float all = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffu, all, d));
          if (lane == 0) *vmax = all;
        }
        __syncwarp();
        if (p.slopes && warp == 1) {
          const int j = tok0 + lane - rq.base;
          int at = tok0 + lane;
          if (j >= 0 && j < rq.n) {
            const uint64_t its = p.tree_mask ? __ldg(p.tree_mask + rq.row0 + j) & all_new : (2ull << j) - 1;
            at = rq.base + __popcll(its & ~(1ull << j));
          }
          pos_k[lane] = at;
        }
        fence_proxy_async();
        tmem_before();
        if (__syncthreads_or(lost)) {
          lost = true;
          break;
        }
        if (tid == 0) {
          tmem_after();
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            umma_ss(tmem + R::kS, smem_desc(smem_u32(sm + R::kQ) + k * 2 * R::kQLbo, R::kQLbo, R::kQSbo),
                    smem_desc(smem_u32(sm + R::kK) + k * 2 * R::kKLbo, R::kKLbo, R::kKSbo), idesc(kMxTile), k > 0);
          umma_commit(smem_u32(bar_s));
        }
        busy_s = true;
        // ---- V, once the previous product has read its operands
        load_codes(sv);
        const float4 ve = *reinterpret_cast<const float4*>(vfac + sub * 16 + 4 * c);   // of this lane's tokens
        if (busy_o) {
          lost |= !mbar_wait_bounded(smem_u32(bar_o), phase_o);
          phase_o ^= 1;
          busy_o = false;
        }
#pragma unroll
        for (int k = 0; k < UB; ++k) {
          uint32_t hv[4][2];   // [channel j][token pair]
          if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
            for (int j = 0; j < 4; ++j) codes_e4m3(edge ? drop_nan_codes(w[k][j]) : w[k][j], hv[j]);
          } else {
            codes_e2m1(w[k][0], hv[0]);
            codes_e2m1(w[k][1], hv[2]);
          }
          const uint32_t z = *reinterpret_cast<const uint32_t*>(sv + mx_scale_off<D, FMT>(sub * 4 + c, b0 + k));
          float y[4] = {ratio(scale_f32(z, 0), ve.x), ratio(scale_f32(z, 1), ve.y), ratio(scale_f32(z, 2), ve.z),
                        ratio(scale_f32(z, 3), ve.w)};
          // (a NaN block's ratio is large: its codes are 0, and so is what it gives)
          const uint32_t s01 = pack_f16(fminf(y[0], 1.f), fminf(y[1], 1.f)), s23 = pack_f16(fminf(y[2], 1.f), fminf(y[3], 1.f));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = 4 * g + j;
            *reinterpret_cast<uint2*>(sm + R::kV + (b0 + k) * R::kVBlock + (r >> 3) * R::kVSbo +
                                      (2 * sub + (c >> 1)) * R::kVLbo + (r & 7) * 16 + (c & 1) * 8) =
                make_uint2(mul_f16(hv[j][0], s01), mul_f16(hv[j][1], s23));
          }
        }
        // ---- scores in log2 units
        lost |= !mbar_wait_bounded(smem_u32(bar_s), phase_s);
        phase_s ^= 1;
        busy_s = false;
        __syncwarp();
        tmem_after();
        float x[32];
        tmem_ld32(mine + R::kS, x);
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < 32; t += 4) {
          const float4 fc = *reinterpret_cast<const float4*>(fac + t);
          const float2 a = mul2(mul2(make_float2(x[t], x[t + 1]), make_float2(f, f)), make_float2(fc.x, fc.y));
          const float2 b = mul2(mul2(make_float2(x[t + 2], x[t + 3]), make_float2(f, f)), make_float2(fc.z, fc.w));
          x[t] = a.x;
          x[t + 1] = a.y;
          x[t + 2] = b.x;
          x[t + 3] = b.y;
        }
        if (p.softcap > 0.f) {
#pragma unroll
          for (int t = 0; t < 32; ++t) x[t] = p.softcap * kLog2e * tanh_abs(x[t]);
        }
        uint32_t vis = ~0u;
        if (edge) {   // bits of the tokens that the row sees
          const int lo = rq.base - tok0;   // the prefix's part of the tile, < 32
          vis = lo > 0 ? ((1u << lo) - 1) | (uint32_t)(sees << lo) : (uint32_t)(lo > -64 ? sees >> -lo : 0ull);
        }
        if (p.slopes) {
#pragma unroll
          for (int t = 0; t < 32; ++t) x[t] -= slope * (float)(pos_q - pos_k[t]);
        }
        if (edge) {
#pragma unroll
          for (int t = 0; t < 32; ++t)
            if (!(vis >> t & 1)) x[t] = -INFINITY;
        }
#pragma unroll
        for (int t = 0; t < 32; ++t) top = fmaxf(top, x[t]);
        if constexpr (NB == 4) {
          const uint4 z = *reinterpret_cast<const uint4*>(vnan);
          poison |= (z.x & vis ? 1u : 0u) | (z.y & vis ? 2u : 0u) | (z.z & vis ? 4u : 0u) | (z.w & vis ? 8u : 0u);
        } else {
          const uint2 z = *reinterpret_cast<const uint2*>(vnan);
          poison |= (z.x & vis ? 1u : 0u) | (z.y & vis ? 2u : 0u);
        }
        // ---- raise the references if a score or a weight could leave its range
        const bool over = top > m + kScoreSlack || ex2(top - (m == -INFINITY ? 0.f : m)) * *vmax * rs > kWeightMax;
        if (__any_sync(0xffffffffu, over)) {   // (all lanes: the TMEM accesses are the warp's)
          const float mn = fmaxf(m, top);
          if (m != -INFINITY) l *= ex2(m - mn);
          m = mn;
          float bm = -INFINITY;
#pragma unroll
          for (int t = 0; t < 32; ++t) bm = fmaxf(bm, x[t] + (float)((__float_as_int(vfac[t]) >> 23) - 127));
          const float Mn = fmaxf(M, bm - kWeightExp);
          const float back = M == -INFINITY ? 0.f : ex2(M - Mn);
          M = Mn;
          rs = Mn == -INFINITY ? 0.f : ex2(mn - Mn);
          if (!first) {
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
              float o[32];
              tmem_ld32(mine + R::kO + 32 * b, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= back;
              tmem_st32(mine + R::kO + 32 * b, o);
            }
          }
        }
        // ---- weights
        {
          const float mi = m == -INFINITY ? 0.f : m;
          const float2 r2 = make_float2(rs, rs);
          float2 sum = make_float2(0.f, 0.f);
          uint32_t pw[16];
#pragma unroll
          for (int t = 0; t < 32; t += 4) {
            const float2 y = make_float2(ex2(x[t] - mi), ex2(x[t + 1] - mi));
            const float2 z = make_float2(ex2(x[t + 2] - mi), ex2(x[t + 3] - mi));
            sum = add2(sum, add2(y, z));
            const float4 sc = *reinterpret_cast<const float4*>(vfac + t);
            const float2 wy = mul2(mul2(y, make_float2(sc.x, sc.y)), r2), wz = mul2(mul2(z, make_float2(sc.z, sc.w)), r2);
            pw[t / 2] = pack_f16(wy.x, wy.y);
            pw[t / 2 + 1] = pack_f16(wz.x, wz.y);
          }
          l += sum.x + sum.y;
          __syncwarp();
          tmem_st16(mine + R::kP, pw);
        }
        tmem_wait_st();
        fence_proxy_async();
        tmem_before();
        if (__syncthreads_or(lost)) {
          lost = true;
          break;
        }
        if (tid == 0) {
          tmem_after();
#pragma unroll
          for (int k = 0; k < 2; ++k)
            umma_ts(tmem + R::kO, tmem + R::kP + 8 * k,
                    smem_desc(smem_u32(sm + R::kV) + k * 2 * R::kVLbo, R::kVLbo, R::kVSbo), idesc(D), !(first && k == 0));
          umma_commit(smem_u32(bar_o));
        }
        busy_o = true;
        first = false;
      } else if (__syncthreads_or(lost)) {
        lost = true;
        break;
      }
      if (issued < count) issue(slot);   // all threads have read the slot
      ++done;
      if (++slot == S) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (lost) break;

    // ------------------------------------------------ the unit's rows, or this block's part of them
    if (busy_o) {
      lost |= !mbar_wait_bounded(smem_u32(bar_o), phase_o);
      phase_o ^= 1;
      busy_o = false;
    }
    if (__syncthreads_or(lost)) {
      lost = true;
      break;
    }
    tmem_after();
    const bool whole = first_tile == 0 && n_tiles == cc.tiles;
    float* part = p.partials + ((size_t)(2 * wid + (first_tile == 0)) * CHUNK + tid) * (D + 4);
    const int64_t at = (int64_t)(rq.row0 + rho / p.G) * p.Hq + h * p.G + rho % p.G;
    if (there) {
      if (!whole) *reinterpret_cast<float2*>(part + D) = make_float2(m, l);
      else if (p.lse) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
    }
    const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float o[32];
      tmem_ld32(mine + R::kO + 32 * b, o);
      // a row that saw only NaN has no M: its l is NaN
      const float fb = poison >> b & 1 ? NAN : M == -INFINITY ? l : ex2(M - m) * inv;
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = first ? 0.f : o[i] * fb;
      if (there && !whole) {
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          *reinterpret_cast<float4*>(part + 32 * b + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      } else if (there) {
        uint32_t z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
          z[i] = *reinterpret_cast<const uint32_t*>(&v);
        }
        uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.out) + at * D + 32 * b);
#pragma unroll
        for (int i = 0; i < 4; ++i) dst[i] = make_uint4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
      }
      __syncwarp();
    }
    if (first_tile == 0 && !whole && tid == 0) {
      // the blocks after this one that hold the unit's other tiles
      const int64_t last = begin + done - n_tiles + cc.tiles - 1, longer = (int64_t)extra * (share + 1);
      const int64_t owner = last < longer ? last / (share + 1) : extra + (last - longer) / share;
      p.headers[wid] = make_int4((int)(owner - wid), rq.row0, h, rho0 << 8 | rows);
    }
    tmem_before();   // O is read before the next unit's product writes it: the next barrier orders them
    if (done < count) mx_next_unit<CHUNK>(p, &cc);
  }
  if (lost) {   // copies and products that are still on their way end before the block does
    if (tid == 0) {
      set_fault(p.fault, LOOPVQ_FAULT_TIMEOUT);
      if (busy_s) mbar_wait_bounded(smem_u32(bar_s), phase_s);
      if (busy_o) mbar_wait_bounded(smem_u32(bar_o), phase_o);
      for (int i = done; i < issued; ++i) mbar_wait_bounded(smem_u32(full + i % S), (uint32_t)(i / S) & 1);
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
  const cudaError_t e =
      cudaFuncSetAttribute(mx_rows_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  mx_rows_kernel<D, FMT><<<grid, kRowsThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

int mx_rows_workers() { return 2 * device_sm_count(); }

cudaError_t mx_rows_launch(int head_dim, int format, const MxAttnParams& p, int grid, cudaStream_t s) {
  if (head_dim == 128)
    return format == LOOPVQ_MX_E4M3 ? launch<128, LOOPVQ_MX_E4M3>(p, grid, s) : launch<128, LOOPVQ_MX_E2M1>(p, grid, s);
  return format == LOOPVQ_MX_E4M3 ? launch<64, LOOPVQ_MX_E4M3>(p, grid, s) : launch<64, LOOPVQ_MX_E2M1>(p, grid, s);
}

}  // namespace loopvq
