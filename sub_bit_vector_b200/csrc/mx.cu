// Microscaled KV cache: quantise as written, read back, keep accepted drafts.
//
// A block of 32 channels of one token shares the scale 2^e, e the least
// integer in [-64, 56] with max|x| <= top * 2^e; a code is the element value
// nearest to x * 2^-e.  Scaling by a power of two is exact, so the one
// rounding is the conversion instruction's (nearest even).
//
// The kernels move bytes; DRAM bounds them.  For many tokens a warp owns one
// tile (32 tokens) of one head of K or V, because a tile's bytes interleave its tokens
// the way the attention's matrix instructions take them: the lane that loads
// a piece of a row in the order of the pool is the lane that stores it, in
// 16-byte pieces, with no exchange but the block's maximum.  The warps of a
// CTA take neighbouring heads, whose rows are neighbours in x.  An 8K prompt of
// 16 heads x 128 and 4 steps, bf16 to e2m1, is written in 67 us (339 MB: 5.1 TB/s;
// the ALU pipe is at two thirds, 12 instructions per 32 elements, most of them
// for the blocks' maxima and scales); a 16K context, e4m3 to bf16, is read in 130
// us (814 MB: 6.25 TB/s, 95% of a copy).  For a few tokens see MxQuad.
#include "mx.cuh"

namespace loopvq {
namespace {

// Up to so many new tokens of a request the kernels for a few tokens run.  128
// requests, e4m3, write and read with tiles / with quads: 1 token 22.7 + 10.9 /
// 6.7 + 4.6 us, 16 tokens 50 + 33 / 35 + 26, 32 tokens 65 + 48 / 65 + 48; but 4
// requests, 16 tokens 8.4 + 5.6 / 9.2 + 6.2, 32 tokens 7.4 + 5.5 / 15 + 9.6, since
// a warp goes through its request's quads one after another.
constexpr int kMxFew = 16;

struct MxMoveParams {
  MxLayout L;
  int H, n_steps, first_step, head_groups;
  bool few;
  int64_t st, sn, sh;
  const void *xk, *xv;   // write: in
  void *ok, *ov;         // read: out
  uint8_t *pk, *pv;
  uint32_t* fault;
};

// Scale byte of a block with largest magnitude bits m, and 2^-e.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale(uint32_t m, float* inv) {
  // top = 1.75 * 2^8 or 1.5 * 2^2: e + 127 = exponent field - 8 (2), one more
  // above top's fraction, which the addition carries
  constexpr uint32_t kTopExp = FMT == LOOPVQ_MX_E4M3 ? 8 : 2;
  constexpr uint32_t kTopFrac = FMT == LOOPVQ_MX_E4M3 ? 0x600000u : 0x400000u;
  const int f = (int)((m + (0x7fffffu - kTopFrac)) >> 23) - (int)kTopExp;
  const uint32_t byte = (uint32_t)max(kMxExpMin + 127, min(kMxExpMax + 127, f));
  *inv = __uint_as_float((254u - byte) << 23);
  return m >= 0x7f800000u ? kMxNan : byte;
}
// Four scaled values to codes: e4m3 in the 4 bytes, e2m1 in the low 4 nibbles.
template <int FMT>
__device__ __forceinline__ uint32_t mx_codes4(float a, float b, float c, float d) {
  if constexpr (FMT == LOOPVQ_MX_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | (uint32_t)hi << 16;
  } else {
    uint16_t r;
    asm("{\n .reg .b8 p0, p1;\n cvt.rn.satfinite.e2m1x2.f32 p0, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 p1, %4, %3;\n"
        " mov.b16 %0, {p0, p1};\n}"
        : "=h"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  }
}

// N consecutive channels; vector stores when VEC.
template <typename T, int N, bool VEC>
__device__ __forceinline__ void store_channels(T* p, const float* v) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (VEC && N == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else if constexpr (VEC) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      if constexpr (VEC)
        reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      else
        for (int j = 0; j < 4; ++j) p[4 * i + j] = v[4 * i + j];
    }
  }
}

// N consecutive channels as they are in memory: two bf16 or one fp32 a word.
template <typename T, int N, bool VEC>
struct MxRaw {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 2) {
          const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + 2 * i;
          w[i] = (uint32_t)q[0] | (uint32_t)q[1] << 16;
        } else {
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
      }
    } else if constexpr (kWords == 2) {
      const uint2 u = ld_once(reinterpret_cast<const uint2*>(p));
      w[0] = u.x; w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 u = ld_once(reinterpret_cast<const uint4*>(p) + i);
        w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // Largest magnitude's bits: 16 of bf16 (compared in pairs), 32 of fp32.
  __device__ __forceinline__ uint32_t peak() const {
    uint32_t m = 0;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
      return max(m & 0xffffu, m >> 16);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (sizeof(T) == 2) return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    else return __uint_as_float(w[i]);
  }
};
// The peaks of CNT blocks over the lanes that differ in the bits FROM .. TO of
// their number, as fp32 bits.  bf16 peaks travel in pairs.
template <typename T, int CNT, int FROM, int TO>
__device__ __forceinline__ void mx_peaks(uint32_t (&m)[CNT]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      uint32_t w = m[i] | m[i + 1] << 16;
#pragma unroll
      for (int d = FROM; d <= TO; d <<= 1) w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, d));
      m[i] = w << 16;
      m[i + 1] = w & 0xffff0000u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
#pragma unroll
      for (int d = FROM; d <= TO; d <<= 1) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], d));
  }
}

// What a warp of the write and read kernels works on.
struct MxUnit {
  MxReq q;
  int tok0;        // first token of the tile
  int kind, h, s;  // K or V, head, step - first_step
  uint8_t* tile;
};
// The unit of this warp, or false if it has none.
template <int D, int FMT>
__device__ __forceinline__ bool mx_unit(const MxMoveParams& p, MxUnit* u) {
  const int hg = blockIdx.x % p.head_groups, tile_i = blockIdx.x / p.head_groups;
  const int hk = hg * 8 + (threadIdx.x >> 5);
  if (hk >= 2 * p.H) return false;
  const int r = blockIdx.z;
  if (!mx_request(p.L, r, &u->q, p.fault)) return false;
  const int t = u->q.base / kMxTile + tile_i;
  u->tok0 = t * kMxTile;
  if (u->q.n == 0 || u->tok0 >= u->q.ctx) return false;
  const int64_t pt = mx_pool_tile(p.L, r, t, p.fault);
  if (pt < 0) return false;
  u->kind = hk >= p.H;
  u->h = hk - u->kind * p.H;
  u->s = blockIdx.y;
  u->tile = (u->kind ? p.pv : p.pk) +
            (((int64_t)(p.first_step + u->s) * p.H + u->h) * p.L.pool_tiles + pt) * MxTile<D, FMT>::kBytes;
  return true;
}

// Quantise: K lanes hold 8 channels of two tokens per block, V lanes 4
// channels of four tokens.
template <int D, int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 3 : 2) mx_write_kernel(const MxMoveParams p) {
  using Tile = MxTile<D, FMT>;
  constexpr int NB = Tile::kBlocks;
  mx_begin();
  MxUnit u;
  if (!mx_unit<D, FMT>(p, &u)) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const T* x = reinterpret_cast<const T*>(u.kind ? p.xv : p.xk) + u.s * p.st + u.h * p.sh +
               (int64_t)u.q.row0 * p.sn;
#pragma unroll 1
  for (int sub = 0; sub < 2; ++sub) {
    const int first = u.tok0 + 16 * sub;
    if (first + 16 <= u.q.base || first >= u.q.ctx) continue;
    if (u.kind == LOOPVQ_KEYS) {
      const int tok[2] = {first + 4 * (g >> 1) + (g & 1), first + 4 * (g >> 1) + (g & 1) + 2};
      const bool in[2] = {tok[0] >= u.q.base && tok[0] < u.q.ctx, tok[1] >= u.q.base && tok[1] < u.q.ctx};
      MxRaw<T, 8, VEC> v[2][NB];
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (in[a]) v[a][b].load(x + (int64_t)(tok[a] - u.q.base) * p.sn + 32 * b + 8 * c);
          else v[a][b].zero();
        }
      uint32_t sc[2] = {0, 0}, lo[2][NB], hi[2][NB];
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        uint32_t m[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) m[b] = v[a][b].peak();
        mx_peaks<T, NB, 1, 2>(m);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float inv;
          const uint32_t byte = mx_scale<FMT>(m[b], &inv);
          sc[a] |= byte << (8 * b);
          const auto& w = v[a][b];
          const uint32_t keep = byte != kMxNan ? ~0u : 0u;
          lo[a][b] = mx_codes4<FMT>(w[0] * inv, w[1] * inv, w[2] * inv, w[3] * inv);
          hi[a][b] = mx_codes4<FMT>(w[4] * inv, w[5] * inv, w[6] * inv, w[7] * inv) & keep;
          if constexpr (FMT == LOOPVQ_MX_E2M1) lo[a][b] |= hi[a][b] << 16;
          lo[a][b] &= keep;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint8_t* d = u.tile + mx_code_off<D, FMT>(sub, b, lane);
        if constexpr (FMT == LOOPVQ_MX_E4M3) {
          if (in[0] && in[1]) {
            *reinterpret_cast<uint4*>(d) = make_uint4(lo[0][b], hi[0][b], lo[1][b], hi[1][b]);
          } else {
            if (in[0]) *reinterpret_cast<uint2*>(d) = make_uint2(lo[0][b], hi[0][b]);
            if (in[1]) *reinterpret_cast<uint2*>(d + 8) = make_uint2(lo[1][b], hi[1][b]);
          }
        } else {
          if (in[0] && in[1]) {
            if ((b & 1) == 0)
              *reinterpret_cast<uint4*>(d) = make_uint4(lo[0][b], lo[1][b], lo[0][b + 1], lo[1][b + 1]);
          } else {
            if (in[0]) *reinterpret_cast<uint32_t*>(d) = lo[0][b];
            if (in[1]) *reinterpret_cast<uint32_t*>(d + 4) = lo[1][b];
          }
        }
      }
      // lane c stores the scales of block c
      if (c < NB) {
        uint8_t* d = u.tile + mx_scale_off<D, FMT>(sub * 4 + (g >> 1), c) + (g & 1);
#pragma unroll
        for (int a = 0; a < 2; ++a)
          if (in[a]) d[2 * a] = (uint8_t)(sc[a] >> (8 * c));
      }
    } else {
      const int tok = first + 4 * c;
      uint32_t in_mask = 0;   // a byte per new token of the quad
      MxRaw<T, 4, VEC> v[4][NB];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const bool in = tok + t >= u.q.base && tok + t < u.q.ctx;
        in_mask |= in ? 0xffu << (8 * t) : 0u;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (in) v[t][b].load(x + (int64_t)(tok + t - u.q.base) * p.sn + 32 * b + 4 * g);
          else v[t][b].zero();
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t m[4], sc = 0, keep = 0;
        float inv[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) m[t] = v[t][b].peak();
        mx_peaks<T, 4, 4, 16>(m);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t byte = mx_scale<FMT>(m[t], &inv[t]);
          sc |= byte << (8 * t);
          keep |= byte == kMxNan ? 0u : (FMT == LOOPVQ_MX_E4M3 ? 0xffu << (8 * t) : 0xfu << (4 * t));
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = mx_codes4<FMT>(v[0][b][j] * inv[0], v[1][b][j] * inv[1], v[2][b][j] * inv[2], v[3][b][j] * inv[3]) & keep;
        uint8_t* d = u.tile + mx_code_off<D, FMT>(sub, b, lane);
        uint32_t* ds = reinterpret_cast<uint32_t*>(u.tile + mx_scale_off<D, FMT>(sub * 4 + c, b));
        if (in_mask == 0) continue;
        // the quad's old tokens keep their bits
        if constexpr (FMT == LOOPVQ_MX_E4M3) {
          uint4 o = make_uint4(w[0], w[1], w[2], w[3]);
          if (in_mask != 0xffffffffu) {
            const uint4 old = *reinterpret_cast<const uint4*>(d);
            o.x = (o.x & in_mask) | (old.x & ~in_mask);
            o.y = (o.y & in_mask) | (old.y & ~in_mask);
            o.z = (o.z & in_mask) | (old.z & ~in_mask);
            o.w = (o.w & in_mask) | (old.w & ~in_mask);
          }
          *reinterpret_cast<uint4*>(d) = o;
        } else {
          uint2 o = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
          if (in_mask != 0xffffffffu) {
            uint32_t nm = 0;   // a nibble per token, twice
#pragma unroll
            for (int t = 0; t < 4; ++t) nm |= (in_mask >> (8 * t) & 1u) ? 0x000f000fu << (4 * t) : 0u;
            const uint2 old = *reinterpret_cast<const uint2*>(d);
            o.x = (o.x & nm) | (old.x & ~nm);
            o.y = (o.y & nm) | (old.y & ~nm);
          }
          *reinterpret_cast<uint2*>(d) = o;
        }
        if (g == 0) *ds = in_mask == 0xffffffffu ? sc : (sc & in_mask) | (*ds & ~in_mask);
      }
    }
  }
}

// Codes to values.
template <int FMT>
__device__ __forceinline__ float2 mx_value2(uint32_t code2) {  // two codes in the low 16 or 8 bits
  uint32_t h;
  if constexpr (FMT == LOOPVQ_MX_E4M3)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code2));
  else
    asm("{\n .reg .b8 a, z1, z2, z3;\n mov.b32 {a, z1, z2, z3}, %1;\n cvt.rn.f16x2.e2m1x2 %0, a;\n}" : "=r"(h) : "r"(code2));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float mx_scale_value(uint32_t byte) {
  // 2^(byte - 127); byte 0 is the subnormal 2^-127, 255 is NaN
  return __uint_as_float(byte == kMxNan ? 0x7fffffffu : byte == 0 ? 0x00400000u : byte << 23);
}

template <int D, int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_read_kernel(const MxMoveParams p) {
  using Tile = MxTile<D, FMT>;
  constexpr int NB = Tile::kBlocks;
  mx_begin();
  MxUnit u;
  if (!mx_unit<D, FMT>(p, &u)) return;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  T* x = reinterpret_cast<T*>(u.kind ? p.ov : p.ok) + u.s * p.st + u.h * p.sh + (int64_t)u.q.row0 * p.sn;
#pragma unroll 1
  for (int sub = 0; sub < 2; ++sub) {
    const int first = u.tok0 + 16 * sub;
    if (first + 16 <= u.q.base || first >= u.q.ctx) continue;
    // the half tile's codes and scales of this lane
    uint32_t w[NB][Tile::kLaneBytes / 4], sw[NB];
    if constexpr (FMT == LOOPVQ_MX_E4M3) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint4 z = ld_once(reinterpret_cast<const uint4*>(u.tile + mx_code_off<D, FMT>(sub, b, lane)));
        w[b][0] = z.x; w[b][1] = z.y; w[b][2] = z.z; w[b][3] = z.w;
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; b += 2) {
        const uint4 z = ld_once(reinterpret_cast<const uint4*>(u.tile + mx_code_off<D, FMT>(sub, b, lane)));
        w[b][0] = z.x; w[b][1] = z.y; w[b + 1][0] = z.z; w[b + 1][1] = z.w;
      }
    }
    if (u.kind == LOOPVQ_KEYS) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        const int tok = first + 4 * (g >> 1) + (g & 1) + 2 * a;
        if (tok < u.q.base || tok >= u.q.ctx) continue;
        T* row = x + (int64_t)(tok - u.q.base) * p.sn;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float s = mx_scale_value(u.tile[mx_scale_off<D, FMT>(sub * 4 + (g >> 1), b) + (g & 1) + 2 * a]);
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = FMT == LOOPVQ_MX_E4M3 ? mx_value2<FMT>(w[b][2 * a + (i >> 1)] >> (16 * (i & 1)))
                                                   : mx_value2<FMT>(w[b][a] >> (8 * i));
            v[2 * i] = f.x * s;
            v[2 * i + 1] = f.y * s;
          }
          store_channels<T, 8, VEC>(row + 32 * b + 8 * c, v);
        }
      }
    } else {
#pragma unroll
      for (int b = 0; b < NB; ++b)
        sw[b] = *reinterpret_cast<const uint32_t*>(u.tile + mx_scale_off<D, FMT>(sub * 4 + c, b));
#pragma unroll
      for (int t2 = 0; t2 < 2; ++t2)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float v[2][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = FMT == LOOPVQ_MX_E4M3 ? mx_value2<FMT>(w[b][j] >> (16 * t2))
                                                   : mx_value2<FMT>(w[b][j >> 1] >> (16 * (j & 1) + 8 * t2));
            v[0][j] = f.x;
            v[1][j] = f.y;
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int tok = first + 4 * c + 2 * t2 + t;
            if (tok < u.q.base || tok >= u.q.ctx) continue;
            const float s = mx_scale_value(sw[b] >> (8 * (2 * t2 + t)) & 255u);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[t][j] *= s;
            store_channels<T, 4, VEC>(x + (int64_t)(tok - u.q.base) * p.sn + 32 * b + 4 * g, v[t]);
          }
        }
    }
  }
}

// ------------------------------------------------------- a few tokens, keep
//
// For a few tokens of each request a tile per warp would move 32 tokens' bytes
// for one.  Here a lane holds 4 channels of the tokens of a quad (4 * i ..
// 4 * i + 3 of a tile): the bytes of a quad that a lane reads or writes are its
// own, so quads with old tokens are merged in registers without exchange.  A
// warp covers 128 channels: one head (D = 128) or two (64).
template <int D, int FMT>
struct MxQuad {
  using Tile = MxTile<D, FMT>;
  uint8_t* tile;
  int sub, c, b, l;   // half, quad of the half, block, lane within the block
  __device__ __forceinline__ MxQuad(uint8_t* tile_, int quad, int lane)
      : tile(tile_), sub(quad >> 2), c(quad & 3), b(lane % (D / 4) >> 3), l(lane & 7) {}
  // K: the 4 codes of token t, 4 or 2 bytes
  __device__ __forceinline__ uint8_t* key(int t) const {
    const int per = Tile::kLaneBytes / 4;
    return tile + mx_code_off<D, FMT>(sub, b, (2 * c + (t & 1)) * 4 + (l >> 1)) + ((t >> 1) * 2 + (l & 1)) * per;
  }
  __device__ __forceinline__ uint32_t load_key(int t) const {
    if constexpr (FMT == LOOPVQ_MX_E4M3) return *reinterpret_cast<const uint32_t*>(key(t));
    else return *reinterpret_cast<const uint16_t*>(key(t));
  }
  __device__ __forceinline__ void store_key(int t, uint32_t w) const {
    if constexpr (FMT == LOOPVQ_MX_E4M3) *reinterpret_cast<uint32_t*>(key(t)) = w;
    else *reinterpret_cast<uint16_t*>(key(t)) = (uint16_t)w;
  }
  // V: [channel j][token t], 16 or 8 bytes
  __device__ __forceinline__ uint8_t* value() const { return tile + mx_code_off<D, FMT>(sub, b, l * 4 + c); }
  __device__ __forceinline__ uint4 load_value() const {
    if constexpr (FMT == LOOPVQ_MX_E4M3) return *reinterpret_cast<const uint4*>(value());
    const uint2 w = *reinterpret_cast<const uint2*>(value());
    return make_uint4(w.x, w.y, 0u, 0u);
  }
  __device__ __forceinline__ void store_value(uint4 w) const {
    if constexpr (FMT == LOOPVQ_MX_E4M3) *reinterpret_cast<uint4*>(value()) = w;
    else *reinterpret_cast<uint2*>(value()) = make_uint2(w.x, w.y);
  }
  // Codes of token t out of a value piece, as load_key gives them.
  static __device__ __forceinline__ uint32_t token(uint4 w, int t) {
    if constexpr (FMT == LOOPVQ_MX_E4M3) {
      const uint32_t lo = __byte_perm(w.x, w.y, t | (4 + t) << 4), hi = __byte_perm(w.z, w.w, t | (4 + t) << 4);
      return __byte_perm(lo, hi, 0x5410);
    } else {
      const uint32_t x = w.x >> (4 * t), y = w.y >> (4 * t);
      return (x & 15u) | (x >> 16 & 15u) << 4 | (y & 15u) << 8 | (y >> 16 & 15u) << 12;
    }
  }
  // A value piece with token t's codes put in.
  static __device__ __forceinline__ uint4 with_token(uint4 w, int t, uint32_t v) {
    if constexpr (FMT == LOOPVQ_MX_E4M3) {
      const uint32_t keep = ~(0xffu << (8 * t));
      w.x = (w.x & keep) | (v & 0xffu) << (8 * t);
      w.y = (w.y & keep) | (v >> 8 & 0xffu) << (8 * t);
      w.z = (w.z & keep) | (v >> 16 & 0xffu) << (8 * t);
      w.w = (w.w & keep) | (v >> 24) << (8 * t);
    } else {
      const uint32_t keep = ~(0x000f000fu << (4 * t));
      w.x = (w.x & keep) | ((v & 15u) | (v >> 4 & 15u) << 16) << (4 * t);
      w.y = (w.y & keep) | ((v >> 8 & 15u) | (v >> 12 & 15u) << 16) << (4 * t);
    }
    return w;
  }
  // Scale byte of token t.
  __device__ __forceinline__ uint8_t* scale(int t) const { return tile + mx_scale_off<D, FMT>(sub * 4 + c, b) + t; }
};

// What a lane of the kernels for a few tokens works on: K and V of a head,
// whose loads are on their way together.
template <int D>
struct MxFew {
  MxReq q;
  int h;
  bool there;
  __device__ __forceinline__ MxFew(const MxLayout& L, int H, uint32_t* fault) {
    constexpr int kHeads = 128 / D;
    const int w = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    h = w * kHeads + (threadIdx.x & 31) / (D / 4);
    there = w < (H + kHeads - 1) / kHeads && mx_request(L, blockIdx.z, &q, fault) && q.n > 0;   // uniform in the warp
  }
};

template <int D, int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_write_few_kernel(const MxMoveParams p) {
  using Quad = MxQuad<D, FMT>;
  mx_begin();
  const MxFew<D> u(p.L, p.H, p.fault);
  if (!u.there) return;
  const int lane = threadIdx.x & 31;
  const bool in_h = u.h < p.H;
  const int h = in_h ? u.h : 0;
  const int64_t xo = blockIdx.y * p.st + h * p.sh + (int64_t)u.q.row0 * p.sn + 4 * (lane % (D / 4));
  const int64_t stream = ((int64_t)(p.first_step + blockIdx.y) * p.H + h) * p.L.pool_tiles;
  for (int quad = u.q.base >> 2; quad * 4 < u.q.ctx; ++quad) {
    MxRaw<T, 4, VEC> v[2][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = quad * 4 + t;
      if (tok < u.q.base || tok >= u.q.ctx) continue;
      v[0][t].load(reinterpret_cast<const T*>(p.xk) + xo + (int64_t)(tok - u.q.base) * p.sn);
      v[1][t].load(reinterpret_cast<const T*>(p.xv) + xo + (int64_t)(tok - u.q.base) * p.sn);
    }
    const int64_t pt = mx_pool_tile(p.L, blockIdx.z, quad >> 3, p.fault);
    if (pt < 0) continue;
    const Quad ak(p.pk + (stream + pt) * MxTile<D, FMT>::kBytes, quad & 7, lane);
    const Quad av(p.pv + (stream + pt) * MxTile<D, FMT>::kBytes, quad & 7, lane);
    uint4 piece = {};
    if (in_h) piece = av.load_value();
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = quad * 4 + t;
      if (tok < u.q.base || tok >= u.q.ctx) continue;
      uint32_t m[2] = {v[0][t].peak(), v[1][t].peak()};
      mx_peaks<T, 2, 1, 4>(m);
      if (!in_h) continue;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        float inv;
        const uint32_t byte = mx_scale<FMT>(m[kind], &inv);
        const auto& w = v[kind][t];
        const uint32_t code = byte == kMxNan ? 0u : mx_codes4<FMT>(w[0] * inv, w[1] * inv, w[2] * inv, w[3] * inv);
        if (kind) piece = Quad::with_token(piece, t, code);
        else ak.store_key(t, code);
        if (ak.l == 0) *(kind ? av : ak).scale(t) = (uint8_t)byte;
      }
    }
    if (in_h) av.store_value(piece);
  }
}

template <int D, int FMT, typename T, bool VEC>
__global__ void __launch_bounds__(256) mx_read_few_kernel(const MxMoveParams p) {
  using Quad = MxQuad<D, FMT>;
  mx_begin();
  const MxFew<D> u(p.L, p.H, p.fault);
  if (!u.there || u.h >= p.H) return;
  const int lane = threadIdx.x & 31;
  const int64_t xo = blockIdx.y * p.st + u.h * p.sh + (int64_t)u.q.row0 * p.sn + 4 * (lane % (D / 4));
  const int64_t stream = ((int64_t)(p.first_step + blockIdx.y) * p.H + u.h) * p.L.pool_tiles;
#pragma unroll 2
  for (int quad = u.q.base >> 2; quad < (u.q.ctx + 3) >> 2; ++quad) {
    const int64_t pt = mx_pool_tile(p.L, blockIdx.z, quad >> 3, p.fault);
    if (pt < 0) continue;
    const Quad ak(p.pk + (stream + pt) * MxTile<D, FMT>::kBytes, quad & 7, lane);
    const Quad av(p.pv + (stream + pt) * MxTile<D, FMT>::kBytes, quad & 7, lane);
    const uint32_t sk = *reinterpret_cast<const uint32_t*>(ak.scale(0)), sv = *reinterpret_cast<const uint32_t*>(av.scale(0));
    const uint4 piece = av.load_value();
    uint32_t w[4] = {};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = quad * 4 + t;
      if (tok >= u.q.base && tok < u.q.ctx) w[t] = ak.load_key(t);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = quad * 4 + t;
      if (tok < u.q.base || tok >= u.q.ctx) continue;
#pragma unroll
      for (int kind = 0; kind < 2; ++kind) {
        constexpr int kBits = FMT == LOOPVQ_MX_E4M3 ? 16 : 8;
        const uint32_t code = kind ? Quad::token(piece, t) : w[t];
        const float2 a = mx_value2<FMT>(code & ((1u << kBits) - 1)), b = mx_value2<FMT>(code >> kBits);
        const float s = mx_scale_value((kind ? sv : sk) >> (8 * t) & 255u);
        const float v[4] = {a.x * s, a.y * s, b.x * s, b.y * s};
        store_channels<T, 4, VEC>(reinterpret_cast<T*>(kind ? p.ov : p.ok) + xo + (int64_t)(tok - u.q.base) * p.sn, v);
      }
    }
  }
}

// Keep.  A warp takes all kept tokens' codes of its channels into shared
// memory, and only then writes them to their places: any order of indices is
// safe, nothing is read after it was overwritten.  128 requests that keep 6 to 12
// of 33 to 64 drafts, 4 steps: 27 us (104 with whole tiles in shared memory): a
// token's value codes lie in a quad's 16-byte pieces, so that 1 KB of sectors is
// touched for its 132 bytes, 110 MB in all.
constexpr int kMxKeepTiles = (kMxMaxTree + kMxTile - 2) / kMxTile + 1;   // that 64 tokens can touch
constexpr int kMxKeepWarps = 2;

struct MxKeepParams {
  MxLayout L;
  int H;
  const int32_t *keep, *n_keep;
  int max_keep, room;   // row length of keep; tokens that the shared memory of a warp holds
  uint8_t *pk, *pv;
  uint32_t* fault;
};

template <int D, int FMT>
__global__ void __launch_bounds__(kMxKeepWarps * 32) mx_keep_kernel(const MxKeepParams p) {
  using Quad = MxQuad<D, FMT>;
  extern __shared__ __align__(16) uint32_t sm_all[];   // per warp: codes [room][K, V][32], scales [room][K, V][4] bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* code = sm_all + warp * p.room * 66;
  uint8_t* scale = reinterpret_cast<uint8_t*>(code + p.room * 64);
  mx_begin();
  const MxFew<D> u(p.L, p.H, p.fault);
  if (!u.there) return;
  const int r = blockIdx.z, nk = ld_once(p.n_keep + r);
  if (nk < 0 || nk > u.q.n || nk > p.max_keep || nk > p.room) {
    set_fault(p.fault, LOOPVQ_FAULT_CTX_RANGE);
    return;
  }
  if (nk == 0) return;
  const bool in_h = u.h < p.H;
  const int64_t stream = ((int64_t)blockIdx.y * p.H + (in_h ? u.h : 0)) * p.L.pool_tiles;
  const int t0 = u.q.base / kMxTile;
  int64_t tile_at[kMxKeepTiles];
#pragma unroll
  for (int i = 0; i < kMxKeepTiles; ++i)
    tile_at[i] = (t0 + i) * kMxTile < u.q.ctx ? mx_pool_tile(p.L, r, t0 + i, p.fault) : -1;
  auto tile_of = [&](int pos) {
    const int i = pos / kMxTile - t0;
    return i == 0 ? tile_at[0] : i == 1 ? tile_at[1] : tile_at[2];
  };
  // sources of tokens lane and lane + 32 (-1: the token stays as it is)
  int from[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    from[k] = -1;
    if (i < nk) {
      const int f = ld_once(p.keep + (int64_t)r * p.max_keep + i);
      if (f < 0 || f >= u.q.n) set_fault(p.fault, LOOPVQ_FAULT_CTX_RANGE);
      else if (f != i && tile_of(u.q.base + f) >= 0) from[k] = f;
    }
  }
#pragma unroll 4
  for (int i = 0; i < nk; ++i) {
    const int f = __shfl_sync(0xffffffffu, i < 32 ? from[0] : from[1], i & 31);
    if (f < 0 || !in_h) continue;
    const int pos = u.q.base + f;
    const int64_t off = (stream + tile_of(pos)) * MxTile<D, FMT>::kBytes;
    const Quad ak(p.pk + off, (pos >> 2) & 7, lane), av(p.pv + off, (pos >> 2) & 7, lane);
    code[i * 64 + lane] = ak.load_key(pos & 3);
    code[i * 64 + 32 + lane] = Quad::token(av.load_value(), pos & 3);
    if (ak.l == 0) {
      scale[i * 8 + (lane >> 3)] = *ak.scale(pos & 3);
      scale[i * 8 + 4 + (lane >> 3)] = *av.scale(pos & 3);
    }
  }
  const uint32_t moved[2] = {__ballot_sync(0xffffffffu, from[0] >= 0), __ballot_sync(0xffffffffu, from[1] >= 0)};
  __syncwarp();
  if (!in_h) return;
  for (int quad = u.q.base >> 2; quad * 4 < u.q.base + nk; ++quad) {
    const int64_t pt = tile_of(quad * 4);
    if (pt < 0) continue;
    const int64_t off = (stream + pt) * MxTile<D, FMT>::kBytes;
    const Quad ak(p.pk + off, quad & 7, lane), av(p.pv + off, quad & 7, lane);
    uint4 piece = av.load_value();
    bool any = false;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int i = quad * 4 + t - u.q.base;
      if (i < 0 || i >= nk || !(moved[i >> 5] >> (i & 31) & 1)) continue;
      any = true;
      ak.store_key(t, code[i * 64 + lane]);
      piece = Quad::with_token(piece, t, code[i * 64 + 32 + lane]);
      if (ak.l == 0) {
        *ak.scale(t) = scale[i * 8 + (lane >> 3)];
        *av.scale(t) = scale[i * 8 + 4 + (lane >> 3)];
      }
    }
    if (any) av.store_value(piece);
  }
}

// Blocks of `warps` warps over the heads.
unsigned few_blocks(const loopvq_mx_desc* d, int warps) {
  const int heads = 128 / d->head_dim, groups = (d->n_heads_kv + heads - 1) / heads;
  return (unsigned)((groups + warps - 1) / warps);
}

loopvq_status move_setup(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout, int32_t first_step,
                         int32_t n_steps, loopvq_dtype dtype, int64_t st, int64_t sn, int64_t sh, const void* poolK,
                         const void* poolV, uint32_t* fault, MxMoveParams* p, dim3* grid) {
  loopvq_status s = mx_check_desc(desc);
  if (s != LOOPVQ_OK) return s;
  s = mx_check_layout(layout, &p->L);
  if (s != LOOPVQ_OK) return s;
  if (mx_pool_bytes(desc, layout->pool_tokens) == 0) return LOOPVQ_ERR_UNSUPPORTED;
  if (first_step < 0 || n_steps < 1 || n_steps > desc->n_loop - first_step) return LOOPVQ_ERR_INVALID_ARG;
  if (dtype != LOOPVQ_F32 && dtype != LOOPVQ_BF16) return LOOPVQ_ERR_INVALID_ARG;
  if (st < 0 || sn < 0 || sh < 0) return LOOPVQ_ERR_INVALID_ARG;
  if (!poolK || !poolV || ((uintptr_t)poolK & 15) || ((uintptr_t)poolV & 15) || ((uintptr_t)fault & 3))
    return LOOPVQ_ERR_INVALID_ARG;
  p->H = desc->n_heads_kv;
  p->n_steps = n_steps;
  p->first_step = first_step;
  p->head_groups = (2 * p->H + 7) / 8;
  p->st = st; p->sn = sn; p->sh = sh;
  p->pk = (uint8_t*)poolK;
  p->pv = (uint8_t*)poolV;
  p->fault = fault;
  // tiles that a request's new tokens can touch
  int64_t tiles = ((int64_t)p->L.max_new + kMxTile - 2) / kMxTile + 1;
  const int64_t all = ((int64_t)p->L.max_ctx + kMxTile - 1) / kMxTile;
  if (tiles > all) tiles = all;
  const int64_t x = tiles * p->head_groups;
  if (x > 0x7fffffffLL || n_steps > 65535) return LOOPVQ_ERR_UNSUPPORTED;
  *grid = dim3((unsigned)x, (unsigned)n_steps, (unsigned)p->L.batch);
  p->few = p->L.max_new <= kMxFew;
  if (p->few) grid->x = few_blocks(desc, 8);
  return LOOPVQ_OK;
}
// Vector loads and stores of 8 bf16 or 4 fp32 channels.
bool vec_ok(const void* a, const void* b, size_t es, const MxMoveParams& p) {
  const uint64_t m = (uint64_t)(uintptr_t)a | (uint64_t)(uintptr_t)b | (uint64_t)p.st * es | (uint64_t)p.sn * es |
                     (uint64_t)p.sh * es;
  return (m & 15) == 0;
}

}  // namespace

loopvq_status mx_check_desc(const loopvq_mx_desc* d) {
  if (!d || d->n_loop < 1 || d->n_heads_kv < 1 || d->n_heads_q < 1 || d->head_dim < 1) return LOOPVQ_ERR_INVALID_ARG;
  if (d->n_heads_q % d->n_heads_kv) return LOOPVQ_ERR_INVALID_ARG;
  if (d->format != LOOPVQ_MX_E4M3 && d->format != LOOPVQ_MX_E2M1) return LOOPVQ_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return LOOPVQ_ERR_UNSUPPORTED;
  if (d->n_heads_kv > 65535 || d->n_heads_q > 65535) return LOOPVQ_ERR_UNSUPPORTED;
  return LOOPVQ_OK;
}

size_t mx_pool_bytes(const loopvq_mx_desc* d, int64_t pool_tokens) {
  const unsigned __int128 n = (unsigned __int128)d->n_loop * d->n_heads_kv * (uint64_t)(pool_tokens / kMxTile) *
                              mx_tile_bytes(d->head_dim, d->format);
  return n < ((unsigned __int128)1 << 63) ? (size_t)n : 0;
}

loopvq_status mx_check_layout(const loopvq_mx_layout* l, MxLayout* o) {
  if (!l || l->batch < 1 || l->batch > 65535 || l->page_tokens < kMxTile || l->page_tokens % kMxTile ||
      l->max_pages < 1 || l->max_ctx_len < 0 || l->max_new < 0 || l->total_new < 0 || l->pool_tokens < kMxTile ||
      l->pool_tokens % kMxTile)
    return LOOPVQ_ERR_INVALID_ARG;
  if (l->max_ctx_len > (int64_t)l->max_pages * l->page_tokens) return LOOPVQ_ERR_INVALID_ARG;
  if (l->max_ctx_len > kMxMaxContext) return LOOPVQ_ERR_UNSUPPORTED;
  if (!l->pages || !l->ctx_len || !l->new_off) return LOOPVQ_ERR_INVALID_ARG;
  if (((uintptr_t)l->pages | (uintptr_t)l->ctx_len | (uintptr_t)l->new_off) & 3) return LOOPVQ_ERR_INVALID_ARG;
  o->batch = l->batch;
  o->page_tokens = l->page_tokens;
  o->max_pages = l->max_pages;
  o->max_ctx = l->max_ctx_len;
  o->max_new = l->max_new;
  o->total_new = l->total_new;
  o->n_pages = l->pool_tokens / l->page_tokens;
  o->pool_tiles = l->pool_tokens / kMxTile;
  o->pages = l->pages;
  o->ctx_len = l->ctx_len;
  o->new_off = l->new_off;
  return LOOPVQ_OK;
}

}  // namespace loopvq

using namespace loopvq;

#define MX_BY_TYPE(KERNEL, GRID, STREAM, P, T, V)                                                     \
  do {                                                                                                \
    if (desc->head_dim == 128) {                                                                      \
      if (desc->format == LOOPVQ_MX_E4M3) st = mx_launch(KERNEL<128, LOOPVQ_MX_E4M3, T, V>, GRID, 256, 0, STREAM, P); \
      else st = mx_launch(KERNEL<128, LOOPVQ_MX_E2M1, T, V>, GRID, 256, 0, STREAM, P);                             \
    } else {                                                                                          \
      if (desc->format == LOOPVQ_MX_E4M3) st = mx_launch(KERNEL<64, LOOPVQ_MX_E4M3, T, V>, GRID, 256, 0, STREAM, P);  \
      else st = mx_launch(KERNEL<64, LOOPVQ_MX_E2M1, T, V>, GRID, 256, 0, STREAM, P);                              \
    }                                                                                                 \
  } while (0)
#define MX_MOVE(KERNEL, DTYPE, A, B)                                                   \
  do {                                                                                 \
    if (DTYPE == LOOPVQ_BF16) {                                                        \
      if (vec_ok(A, B, 2, p)) MX_BY_TYPE(KERNEL, grid, (cudaStream_t)stream, p, __nv_bfloat16, true);  \
      else MX_BY_TYPE(KERNEL, grid, (cudaStream_t)stream, p, __nv_bfloat16, false);    \
    } else {                                                                           \
      if (vec_ok(A, B, 4, p)) MX_BY_TYPE(KERNEL, grid, (cudaStream_t)stream, p, float, true);          \
      else MX_BY_TYPE(KERNEL, grid, (cudaStream_t)stream, p, float, false);            \
    }                                                                                  \
  } while (0)

extern "C" size_t loopvq_mx_pool_bytes(const loopvq_mx_desc* desc, int64_t pool_tokens) {
  if (mx_check_desc(desc) != LOOPVQ_OK || pool_tokens < kMxTile || pool_tokens % kMxTile) return 0;
  return mx_pool_bytes(desc, pool_tokens);
}

extern "C" loopvq_status loopvq_mx_write(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout,
                                         int32_t first_step, int32_t n_steps, const void* k, const void* v,
                                         loopvq_dtype x_dtype, int64_t stride_t, int64_t stride_n,
                                         int64_t stride_h, void* poolK, void* poolV, uint32_t* fault_bits,
                                         loopvq_stream_t stream) {
  MxMoveParams p = {};
  dim3 grid;
  const loopvq_status bad = move_setup(desc, layout, first_step, n_steps, x_dtype, stride_t, stride_n, stride_h,
                                      poolK, poolV, fault_bits, &p, &grid);
  if (bad != LOOPVQ_OK) return bad;
  cudaError_t st = cudaSuccess;
  if (layout->total_new == 0 || layout->max_new == 0 || layout->max_ctx_len == 0) return LOOPVQ_OK;
  const uintptr_t es = x_dtype == LOOPVQ_BF16 ? 2 : 4;
  if (!k || !v || (uintptr_t)k % es || (uintptr_t)v % es) return LOOPVQ_ERR_INVALID_ARG;
  p.xk = k;
  p.xv = v;
  if (p.few) MX_MOVE(mx_write_few_kernel, x_dtype, k, v);
  else MX_MOVE(mx_write_kernel, x_dtype, k, v);
  return st == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}

extern "C" loopvq_status loopvq_mx_read(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout,
                                        int32_t first_step, int32_t n_steps, const void* poolK, const void* poolV,
                                        void* k_out, void* v_out, loopvq_dtype out_dtype, int64_t stride_t,
                                        int64_t stride_n, int64_t stride_h, uint32_t* fault_bits,
                                        loopvq_stream_t stream) {
  MxMoveParams p = {};
  dim3 grid;
  const loopvq_status bad = move_setup(desc, layout, first_step, n_steps, out_dtype, stride_t, stride_n, stride_h,
                                      poolK, poolV, fault_bits, &p, &grid);
  if (bad != LOOPVQ_OK) return bad;
  cudaError_t st = cudaSuccess;
  if (layout->total_new == 0 || layout->max_new == 0 || layout->max_ctx_len == 0) return LOOPVQ_OK;
  const uintptr_t es = out_dtype == LOOPVQ_BF16 ? 2 : 4;
  if (!k_out || !v_out || (uintptr_t)k_out % es || (uintptr_t)v_out % es) return LOOPVQ_ERR_INVALID_ARG;
  // rows, heads and steps must not meet in the output
  if ((n_steps > 1 && stride_t == 0) || (layout->total_new > 1 && stride_n == 0) ||
      (desc->n_heads_kv > 1 && stride_h == 0))
    return LOOPVQ_ERR_INVALID_ARG;
  p.ok = k_out;
  p.ov = v_out;
  if (p.few) MX_MOVE(mx_read_few_kernel, out_dtype, k_out, v_out);
  else MX_MOVE(mx_read_kernel, out_dtype, k_out, v_out);
  return st == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}

extern "C" loopvq_status loopvq_mx_keep(const loopvq_mx_desc* desc, const loopvq_mx_layout* layout,
                                        const int32_t* keep, const int32_t* n_keep, int32_t max_keep, void* poolK,
                                        void* poolV, uint32_t* fault_bits, loopvq_stream_t stream) {
  MxKeepParams p = {};
  loopvq_status st = mx_check_desc(desc);
  if (st != LOOPVQ_OK) return st;
  st = mx_check_layout(layout, &p.L);
  if (st != LOOPVQ_OK) return st;
  if (mx_pool_bytes(desc, layout->pool_tokens) == 0) return LOOPVQ_ERR_UNSUPPORTED;
  if (!keep || !n_keep || max_keep < 1 || ((uintptr_t)keep & 3) || ((uintptr_t)n_keep & 3)) return LOOPVQ_ERR_INVALID_ARG;
  if (!poolK || !poolV || ((uintptr_t)poolK & 15) || ((uintptr_t)poolV & 15) || ((uintptr_t)fault_bits & 3))
    return LOOPVQ_ERR_INVALID_ARG;
  if (layout->max_new > kMxMaxTree || desc->n_loop > 65535) return LOOPVQ_ERR_UNSUPPORTED;
  if (layout->total_new == 0 || layout->max_new == 0 || layout->max_ctx_len == 0) return LOOPVQ_OK;
  p.H = desc->n_heads_kv;
  p.keep = keep;
  p.n_keep = n_keep;
  p.max_keep = max_keep;
  p.pk = (uint8_t*)poolK;
  p.pv = (uint8_t*)poolV;
  p.fault = fault_bits;
  const dim3 grid(few_blocks(desc, kMxKeepWarps), desc->n_loop, p.L.batch);
  p.room = max_keep < layout->max_new ? max_keep : layout->max_new;
  const size_t smem = (size_t)kMxKeepWarps * p.room * 66 * sizeof(uint32_t);   // at most 33,792 bytes
  auto kfn = desc->head_dim == 128
                 ? (desc->format == LOOPVQ_MX_E4M3 ? mx_keep_kernel<128, LOOPVQ_MX_E4M3> : mx_keep_kernel<128, LOOPVQ_MX_E2M1>)
                 : (desc->format == LOOPVQ_MX_E4M3 ? mx_keep_kernel<64, LOOPVQ_MX_E4M3> : mx_keep_kernel<64, LOOPVQ_MX_E2M1>);
  return mx_launch(kfn, grid, kMxKeepWarps * 32, smem, (cudaStream_t)stream, p) == cudaSuccess ? LOOPVQ_OK : LOOPVQ_ERR_CUDA;
}
