// Attention over the microscaled KV cache: what its kernels share.
#pragma once

#include "mx.cuh"

namespace loopvq {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kScoreSlack = 10.f, kWeightMax = 32768.f, kWeightExp = 8.f;

struct MxAttnParams {
  MxLayout L;
  int H, Hq, G;
  const uint8_t *pk, *pv;   // this loop step's pools
  const void* q;
  int q_bf16, q_vec;
  int64_t qn, qh;
  const uint64_t* tree_mask;
  float scale;   // a quarter (no product overflows) of softmax_scale, times log2 e unless a cap wants natural units
  float softcap, inv_cap, inv_cap2;   // inv_cap: 1 / softcap, at most 2^126; inv_cap2 = 2 log2(e) inv_cap
  const float* slopes;
  void* out;
  int out_bf16;
  float* lse;
  // A worker is a warp (mx_attn_kernel) or a block (mx_rows_kernel).
  int n_workers;
  int4* headers;     // per worker: the unit that starts in it and goes on
  float* partials;   // per worker: 2 slots (a unit that began earlier; one that goes on) of [chunk][D + 4]
  uint32_t* fault;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh y = 1 - 2 / (1 + e^2y), right to 2^-22 absolutely; y2 = 2 log2(e) y.
__device__ __forceinline__ float tanh_abs(float y2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(y2)));
  return fmaf(-2.f, r, 1.f);
}
// Score s, capped, in log2 units.  tanh_abs misses s by 2^-22 of the cap, however
// small s is: with a cap up to kFastCap by 2^-16, 1/32 of what the rounding of a
// weight to fp16 loses.  Above, and with fp32 in or out, tanhf, whose error is
// relative to s (s / cap in steps of 2^-149, s of 2^-21 at most).  64-node tree over
// 32K: 138 us with tanh_abs, 162 with tanhf; chosen per score in one kernel instead of
// in instances of their own (EXACT) 218, since both are computed then.
constexpr float kFastCap = 64.f;
__device__ __forceinline__ float capped_fast(float s, float cap, float inv2) { return cap * kLog2e * tanh_abs(s * inv2); }
__device__ __forceinline__ float capped(float s, float cap, float inv) { return cap * tanhf(s * inv) * kLog2e; }
// 8 channels of a query row.
template <typename T>
__device__ __forceinline__ void load_query(const void* q, int64_t at, int vec, float* v) {
  const T* x = reinterpret_cast<const T*>(q) + at;
  if (!vec) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = to_f32<T>(x[k]);
    return;
  }
  __align__(16) uint32_t w[sizeof(T) * 2];
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k)
    reinterpret_cast<uint4*>(w)[k] = ld_once(reinterpret_cast<const uint4*>(x) + k);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    v[k] = sizeof(T) == 4 ? __uint_as_float(w[k % (sizeof(T) * 2)]) : k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
}
__device__ __forceinline__ uint64_t pair(float2 a) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)));
  return unpair(r);
}
__device__ __forceinline__ void fma2(float* c, float2 a, float2 b) {   // c[0..1] += a * b
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair(a)), "l"(pair(b)), "l"(pair(make_float2(c[0], c[1]))));
  const float2 v = unpair(r);
  c[0] = v.x;
  c[1] = v.y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }
// The 4 codes (e4m3) or 8 (e2m1) of a word as fp16 pairs.
__device__ __forceinline__ void codes_e4m3(uint32_t w, uint32_t* h) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
}
__device__ __forceinline__ void codes_e2m1(uint32_t w, uint32_t* h) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Scale byte t of a word as 2^e (255: infinity, which codes of 0 turn into NaN).
__device__ __forceinline__ float scale_f32(uint32_t w, int t) {
  return __uint_as_float(t == 3 ? (w >> 1) & 0x7f800000u : (w << (23 - 8 * t)) & 0x7f800000u);
}
// e4m3 NaN codes to 0.
__device__ __forceinline__ uint32_t drop_nan_codes(uint32_t w) {
  const uint32_t m = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
  return w & ~((m >> 7) * 0xffu);
}

// Where in the list of tiles a worker is.
struct MxCursor {
  int r, u, units, t, tiles;   // request, unit of its H * chunks, tile of its ctx
};
// Units and tiles of request r (0 units if it has no part in the call).
template <int CHUNK>
__device__ __forceinline__ int mx_units(const MxAttnParams& p, int r, int* tiles) {
  MxReq q;
  *tiles = 0;
  if (!mx_request(p.L, r, &q, p.fault) || q.n == 0 || q.n > kMxMaxTree) return 0;
  *tiles = (q.ctx + kMxTile - 1) / kMxTile;
  return (q.n * p.G + CHUNK - 1) / CHUNK * p.H;
}
// The cursor at tile `at` of the whole list (0 <= at < total); uniform in the
// warp.  u0, t0: units and tiles of request `lane`.
template <int CHUNK>
__device__ __forceinline__ MxCursor mx_seek(const MxAttnParams& p, int64_t at, int u0, int t0, int lane) {
  MxCursor c = {0, 0, 0, 0, 1};
  for (int r0 = 0; r0 < p.L.batch; r0 += 32) {
    int tiles = t0, units = u0;
    if (r0) {
      units = tiles = 0;
      if (r0 + lane < p.L.batch) units = mx_units<CHUNK>(p, r0 + lane, &tiles);
    }
    int64_t sum = (int64_t)units * tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    const int64_t all = __shfl_sync(0xffffffffu, sum, 31);
    if (at < all) {
      const int l = __ffs(__ballot_sync(0xffffffffu, at < sum)) - 1;
      c.r = r0 + l;
      c.units = __shfl_sync(0xffffffffu, units, l);
      c.tiles = __shfl_sync(0xffffffffu, tiles, l);
      const int64_t in = at - (__shfl_sync(0xffffffffu, sum, l) - (int64_t)c.units * c.tiles);
      c.u = (int)(in / c.tiles);
      c.t = (int)(in % c.tiles);
      return c;
    }
    at -= all;
  }
  return c;
}
// On to the next unit; the caller knows that there is one (lengths that
// change under the kernel are the caller's error; indices stay in range).
template <int CHUNK>
__device__ __forceinline__ void mx_next_unit(const MxAttnParams& p, MxCursor* c) {
  c->t = 0;
  if (++c->u < c->units) return;
  c->u = 0;
  do {
    if (++c->r >= p.L.batch) {
      c->r = p.L.batch - 1;
      c->units = p.H;
      c->tiles = 1;
      return;
    }
    c->units = mx_units<CHUNK>(p, c->r, &c->tiles);
  } while (c->units == 0);
}

// The attention of requests with many rows, on the tcgen05 tensor cores (csrc/mx_rows.cu).
constexpr int kMxRowsChunk = 128;
int mx_rows_workers();
cudaError_t mx_rows_launch(int head_dim, int format, const MxAttnParams& p, int grid, cudaStream_t s);

}  // namespace loopvq
