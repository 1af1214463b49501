// Microscaled KV cache: tile layout, request and page lookup shared by the
// kernels that write, read, move and attend over it.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace loopvq {

constexpr int kMxTile = 32;    // tokens of a tile
constexpr int kMxBlock = 32;   // channels that share a scale
constexpr int kMxMaxTree = 64; // new tokens a request may have in attention and keep
constexpr int kMxMaxContext = 0x7fffffff - 128;   // positions up to three tiles past a context's last stay ints
constexpr int kMxExpMin = -64, kMxExpMax = 56;
constexpr uint32_t kMxNan = 255;

// D channels, FMT element format: sizes of one tile.  A unit is 512 bytes,
// 16 per lane: one block of 16 tokens for e4m3, two for e2m1.
template <int D, int FMT>
struct MxTile {
  static constexpr int kBlocks = D / kMxBlock;
  static constexpr int kLaneBytes = FMT == LOOPVQ_MX_E4M3 ? 16 : 8;  // of one block of one half tile
  static constexpr int kHalfBytes = kBlocks * 32 * kLaneBytes;
  static constexpr int kScaleOff = 2 * kHalfBytes;
  static constexpr int kBytes = kScaleOff + kMxTile * kBlocks;
};
// Byte of lane `lane`'s codes of block b of half sub.
template <int D, int FMT>
__host__ __device__ constexpr int mx_code_off(int sub, int b, int lane) {
  return FMT == LOOPVQ_MX_E4M3 ? sub * MxTile<D, FMT>::kHalfBytes + (b * 32 + lane) * 16
                               : sub * MxTile<D, FMT>::kHalfBytes + ((b >> 1) * 32 + lane) * 16 + (b & 1) * 8;
}
// Byte of the scale word of block b for tokens 4 * quad .. 4 * quad + 3 of a tile.
template <int D, int FMT>
__host__ __device__ constexpr int mx_scale_off(int quad, int b) {
  return MxTile<D, FMT>::kScaleOff + (quad * MxTile<D, FMT>::kBlocks + b) * 4;
}
inline size_t mx_tile_bytes(int D, int fmt) {
  return (size_t)kMxTile * D * (fmt == LOOPVQ_MX_E4M3 ? 8 : 4) / 8 + (size_t)kMxTile * (D / kMxBlock);
}

// Loads of what an earlier kernel of the stream may have written, the caller's
// arrays among it.  A kernel may be resident while that kernel still runs
// (mx_begin), so the read-only path, for data that nothing writes while the kernel
// lives, is not for them.  Each load is done once: a checked index stays the one
// that was checked.
__device__ __forceinline__ int32_t ld_once(const int32_t* p) {
  int32_t v;
  asm volatile("ld.global.s32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float ld_once(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint64_t ld_once(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.global.u64 %0, [%1];" : "=l"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_once(const uint2* p) {
  uint2 v;
  asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

struct MxLayout {
  int batch, page_tokens, max_pages, max_ctx, max_new, total_new;
  int64_t n_pages;      // whole pages of the pool
  int64_t pool_tiles;   // tiles of one (step, head)
  const int32_t *pages, *ctx_len, *new_off;
};

struct MxReq {
  int ctx, n, base, row0;  // context, new tokens, first new position, first packed row
};
// Request r's lengths; false (and the fault bit) if they are out of bounds.
__device__ __forceinline__ bool mx_request(const MxLayout& L, int r, MxReq* q, uint32_t* fault) {
  const int ctx = ld_once(L.ctx_len + r), a = ld_once(L.new_off + r), b = ld_once(L.new_off + r + 1);
  const bool ok = a >= 0 && b >= a && b <= L.total_new && b - a <= L.max_new && ctx >= b - a && ctx <= L.max_ctx;
  if (!ok) {
    set_fault(fault, LOOPVQ_FAULT_CTX_RANGE);
    return false;
  }
  q->ctx = ctx;
  q->n = b - a;
  q->base = ctx - q->n;
  q->row0 = a;
  return true;
}
// Pool tile of tile t (tokens 32t ..) of request r, or -1 (and the fault
// bit) for a page id outside the pool.  The caller has 32t < ctx_len.
__device__ __forceinline__ int64_t mx_pool_tile(const MxLayout& L, int r, int t, uint32_t* fault) {
  const int per = L.page_tokens / kMxTile;
  const int id = ld_once(L.pages + (int64_t)r * L.max_pages + t / per);
  if (id < 0 || id >= L.n_pages) {
    set_fault(fault, LOOPVQ_FAULT_POOL_RANGE);
    return -1;
  }
  return (int64_t)id * per + t % per;
}

// The kernels of a step follow one another closely: each may be launched while
// the one before it ends.  Nothing is read or written, and no kernel after this
// one is let in, before that one has ended.
__device__ __forceinline__ void mx_begin() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename K, typename P>
cudaError_t mx_launch(K kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const P& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Host checks shared by the entry points.
loopvq_status mx_check_desc(const loopvq_mx_desc* d);
loopvq_status mx_check_layout(const loopvq_mx_layout* l, MxLayout* out);
// Bytes of a pool of a checked descriptor; 0 if offsets into it would pass 63 bits.
size_t mx_pool_bytes(const loopvq_mx_desc* d, int64_t pool_tokens);

}  // namespace loopvq
