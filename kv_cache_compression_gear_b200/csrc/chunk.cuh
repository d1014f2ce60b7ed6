// chunk.cuh -- attention of chunks of new tokens over a compressed cache: the
// work plan shared by the kernels, and their launches.
//
// Sequence i brings n[i] new tokens. For kv head h its query rows are numbered
// r = token * hq + query head of the group, and cut into units of R rows. A unit
// attends over the row's cached tokens (compressed, then buffered: base[i] of
// them) and over the chunk's own tokens up to its last row's, in tiles of 96.
// All units' tiles are laid end to end (sequence, head, row block), each unit's
// behind `pad` numbers without a tile that stand for its beginning and end, and
// every CTA takes an equal run of `seg` numbers; the part of a unit inside one run
// is a segment. Segments of a unit that no single CTA covers leave partial rows (max,
// sum, accumulator) which chunk_combine or chunk_join merges.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "decode.cuh"

namespace gear {

constexpr int kChunkTile = 96;     // tokens per tile (three groups of 32)
constexpr int kChunkSeqs = 96;     // sequences per launch, at most
constexpr int kChunkTiles = 4096;  // tiles of a launch with long chunks, all its sequences' together, unless one alone has
                                   // more (bounds the scratch of rebuilt tiles)
constexpr int64_t kChunkNumbers = int64_t(1) << 30;   // tile numbers per launch, at most (32-bit with the last run's end)
constexpr int kImgBytes = 64640;   // a rebuilt tile (chunk_tc.cuh)
constexpr int kRowsUnit = 256;     // rows of a unit of paired row tiles
constexpr int kPartRow = 132;      // floats of a partial row: max, sum, 2 unused, acc[128]

struct ChunkArgs {
  CacheView K, V;
  int32_t dtype, B, H, Hq, hq;
  int32_t bits, g, G, W, k, r_max;
  int32_t meta_f16, kc, ch_slots;
  int32_t glog, krecip;      // log2(g); ceil(2^16 / k)
  int32_t n_max, nblk_max, n_b;
  int32_t blk0_rank, buffer_rank;
  int32_t page_tokens, ppr, num_pages, plog;   // plog: log2 of page_tokens, -1 if that is no power of two
  const int32_t* table;      // null: contiguous
  const int32_t* plen;       // [B] or null: real tokens at the head of block 0
  float scale_log2;
  const void* q;             // token t, head j at q + t * qs + j * 128
  const void* kn;            // null: the chunk has no keys of its own
  const void* vn;
  int64_t qs, ks, vs;
  void* out;                 // [T][Hq][128]
  int32_t out_dtype;
  int32_t* status;           // the device error word
  float* part;               // partial rows: [rows of this launch][slots][kPartRow]; of paired row tiles, where only units
                             // of several runs leave some, [ctas][the unit a run goes on with, the one it begins][rows]
  int32_t* join;             // [ctas][8]: the unit that a CTA begins and others end (tiles 0: none)
  // plan
  int32_t nseq, R, pad, seg, slots, par;   // par: partial rows per segment (2: tiles alternate between two accumulators)
  int32_t ctas, small;                // small: at most 32 query rows per unit
  int32_t row[kChunkSeqs], tok0[kChunkSeqs], n[kChunkSeqs];
  int32_t b0[kChunkSeqs], ncomp[kChunkSeqs], nbuf[kChunkSeqs];
  int32_t tile0[kChunkSeqs + 1];      // first tile of each sequence
  // rebuilt tiles: where units of several row blocks read every tile many times, the tiles are
  // rebuilt once, each in kImgBytes of the workspace (null: as they are needed)
  uint8_t* img;
  int32_t sms;
  int32_t img0[kChunkSeqs + 1];       // first rebuilt tile of each sequence; all zero without
};

// Keys of the unit of rows [t R, (t + 1) R) of sequence i, in tiles.
__host__ __device__ inline int chunk_unit_keys(const ChunkArgs& a, int i, int t) {
  const int rows = a.n[i] * a.hq;
  const int last = (t + 1) * a.R < rows ? (t + 1) * a.R : rows;
  return a.ncomp[i] + a.nbuf[i] + (a.kn ? (last - 1) / a.hq + 1 : 0);
}
__host__ __device__ inline int chunk_unit_tiles(const ChunkArgs& a, int i, int t) {
  return (chunk_unit_keys(a, i, t) + kChunkTile - 1) / kChunkTile;
}
__host__ __device__ inline int chunk_blocks(const ChunkArgs& a, int i) { return (a.n[i] * a.hq + a.R - 1) / a.R; }

struct ChunkUnit {
  int i, h, t;      // sequence, kv head, row block
  int tile;         // first tile of the unit in the launch's numbering (behind its pad)
  int tiles;        // tiles of the unit
};

// The unit that number x belongs to (a tile, or one of its pad).
__device__ __forceinline__ ChunkUnit chunk_find(const ChunkArgs& a, int x) {
  int lo = 0, hi = a.nseq;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.tile0[m] <= x) lo = m;
    else hi = m;
  }
  ChunkUnit u;
  u.i = lo;
  const int per = (a.tile0[lo + 1] - a.tile0[lo]) / a.H;
  u.h = (x - a.tile0[lo]) / per;
  u.tile = a.tile0[lo] + u.h * per;
  // row block by row block; tok + rem / hq: tokens up to the block's last row (no division)
  const int rows = a.n[lo] * a.hq, base = a.ncomp[lo] + a.nbuf[lo];
  const int dq = a.R / a.hq, dr = a.R - dq * a.hq;
  int tok = (a.R - 1) / a.hq, rem = (a.R - 1) - tok * a.hq;
  for (u.t = 0;; ++u.t) {
    const int own = a.kn ? ((u.t + 1) * a.R < rows ? tok + 1 : a.n[lo]) : 0;
    u.tiles = (base + own + kChunkTile - 1) / kChunkTile;
    u.tile += a.pad;
    if (x < u.tile + u.tiles) return u;
    u.tile += u.tiles;
    tok += dq;
    rem += dr;
    if (rem >= a.hq) rem -= a.hq, ++tok;
  }
}

// The unit after u (there is one: the caller has numbers left).
__device__ __forceinline__ ChunkUnit chunk_next(const ChunkArgs& a, ChunkUnit u) {
  u.tile += u.tiles + a.pad;
  if (++u.t == chunk_blocks(a, u.i)) {
    u.t = 0;
    if (++u.h == a.H) {
      u.h = 0;
      do ++u.i;
      while (a.tile0[u.i + 1] == a.tile0[u.i]);
    }
  }
  u.tiles = chunk_unit_tiles(a, u.i, u.t);
  return u;
}

// Fills the plan fields of `a` (sequences set) for a device of num_sms SMs.
// slots: the most partial rows that a query row can get.
// False where the numbers do not fit (kChunkNumbers).
bool chunk_plan(ChunkArgs& a, int num_sms);
size_t chunk_workspace_bytes(const ChunkArgs& a);
// tensor-core kernels of 16-bit caches (chunk_f16.cu, chunk_bf16.cu; per-channel key groups: chunk_kc.cu)
cudaError_t chunk_tc_launch_f16(const ChunkArgs& a, cudaStream_t st);
cudaError_t chunk_tc_launch_bf16(const ChunkArgs& a, cudaStream_t st);
cudaError_t chunk_tc_launch_kc(const ChunkArgs& a, cudaStream_t st);
cudaError_t chunk_launch(ChunkArgs& a, cudaStream_t st);   // sets a.join and a.img

}  // namespace gear
