// chunk.cu -- attention of chunks of new tokens over a compressed cache: the
// plan, the kernel of binary32 caches and the merge of partial rows.
//
//   out[j] = sum_t p_t V_t / sum_t p_t,  p_t = exp(tau q_j . K_t),
// over the row's cached tokens (reconstructed: code * scale + zero + L Rf^T,
// outlier slots replaced by their values), its buffer, and the chunk's own
// tokens 0 .. j. One pass over the tokens with a running maximum and sum.
#include <string.h>

#include "chunk.cuh"
#include "common.cuh"

namespace gear {

template <typename T>
__device__ __forceinline__ float elem(const void* p, int64_t i) {
  if constexpr (sizeof(T) == 4) return reinterpret_cast<const float*>(p)[i];
  else if constexpr (std::is_same<T, __half>::value) return __half2float(reinterpret_cast<const __half*>(p)[i]);
  else return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
}

// Channel c of token t of the unit's sequence: compressed, buffered or the chunk's own.
template <typename T, int BITS>
__device__ __forceinline__ float chunk_value(const ChunkArgs& a, const CacheView& C, const void* nw, int64_t ns, int kc,
                                             int i, int h, int t, int c) {
  const int b = a.row[i], nc = a.ncomp[i];
  const int64_t unit = (int64_t)b * a.H + h;
  if (t >= nc) {
    const int j = t - nc;
    if (j < a.nbuf[i]) return elem<T>(C.buf, (unit * a.n_b + j) * 128 + c);
    return elem<T>(nw, (int64_t)(a.tok0[i] + j - a.nbuf[i]) * ns + h * 128 + c);
  }
  int64_t row;
  if (a.table) {
    int pg = __ldg(a.table + (int64_t)b * a.ppr + t / a.page_tokens);
    pg = min(max(pg, 0), a.num_pages - 1);
    row = ((int64_t)pg * a.H + h) * a.page_tokens + t % a.page_tokens;
  } else {
    row = unit * a.n_max + t;
  }
  for (int o = 0; o < a.k; ++o)
    if (C.oidx[row * a.k + o] == c) return elem<T>(C.oval, row * a.k + o);
  constexpr int kPerWord = 32 / BITS;
  const uint32_t code = (C.codes[row * a.W + c / kPerWord] >> (BITS * (c % kPerWord))) & ((1u << BITS) - 1u);
  const int b0 = a.b0[i], blk = t < b0 ? 0 : 1 + (t - b0) / a.n_b;
  float2 sz;
  if (kc) {
    const int slot = t < b0 ? t / a.g : (b0 + a.g - 1) / a.g + (t - b0) / a.g;
    sz = reinterpret_cast<const float2*>(C.meta)[(unit * a.ch_slots + slot) * 128 + c];
  } else {
    sz = a.meta_f16 ? __half22float2(reinterpret_cast<const __half2*>(C.meta)[row * a.G + c / a.g])
                    : reinterpret_cast<const float2*>(C.meta)[row * a.G + c / a.g];
  }
  float v = fmaf((float)code, sz.x, sz.y);
  const int rank = blk == 0 ? a.blk0_rank : a.buffer_rank;
  const float* rf = C.rfac + ((unit * a.nblk_max + blk) * 128 + c) * rpad_of(a.r_max);
  for (int j = 0; j < rank; ++j) {
    const float lv = sizeof(T) == 4 ? reinterpret_cast<const float*>(C.lfac)[row * a.r_max + j]
                                    : __half2float(reinterpret_cast<const __half*>(C.lfac)[row * a.r_max + j]);
    v = fmaf(lv, rf[j], v);
  }
  return v;
}

// R = 8 query rows per unit, 128 threads: thread = channel when a sub-tile of 32
// tokens is rebuilt into shared memory and when it is weighed into the outputs,
// lane = token in the scores and the softmax.
constexpr int kSimtRows = 8;

template <typename T, int BITS>
__global__ void __launch_bounds__(128) chunk_simt(const __grid_constant__ ChunkArgs a) {
  __shared__ float sq[kSimtRows][128], sk[32][129], sv[32][128], sp[kSimtRows][32], sc[kSimtRows], sl[kSimtRows],
      sm[kSimtRows];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int total = a.tile0[a.nseq];
  const int end = min(total, (int)(blockIdx.x + 1) * a.seg);
  for (int x = blockIdx.x * a.seg; x < end;) {
    const ChunkUnit u = chunk_find(a, x);
    x = max(x, u.tile);
    if (x >= end) break;
    const int i = u.i, h = u.h, rows = a.n[i] * a.hq, r0 = u.t * a.R;
    const int nr = min(a.R, rows - r0);
    const int base = a.ncomp[i] + a.nbuf[i], keys = chunk_unit_keys(a, i, u.t);
    const int x1 = min(end, u.tile + u.tiles);
    const int plen = a.plen ? min(max(__ldg(a.plen + a.row[i]), 0), a.b0[i]) : a.b0[i];
    __syncthreads();
    for (int r = 0; r < nr; ++r) {
      const int64_t t = a.tok0[i] + (r0 + r) / a.hq;
      sq[r][tid] = elem<T>(a.q, t * a.qs + (h * a.hq + (r0 + r) % a.hq) * 128 + tid);
    }
    if (tid < kSimtRows) sm[tid] = -INFINITY, sl[tid] = 0.0f;
    float acc[kSimtRows];
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) acc[r] = 0.0f;
    const int t1 = min(keys, (x1 - u.tile) * kChunkTile);
    for (int t0 = (x - u.tile) * kChunkTile; t0 < t1; t0 += 32) {
      const int nt = min(32, t1 - t0);
      __syncthreads();
      for (int j = 0; j < nt; ++j) {
        // padded prompt tokens take no part: their values are not read
        const bool pad = t0 + j >= plen && t0 + j < a.b0[i];
        sk[j][tid] = pad ? 0.0f : chunk_value<T, BITS>(a, a.K, a.kn, a.ks, a.kc, i, h, t0 + j, tid);
        sv[j][tid] = pad ? 0.0f : chunk_value<T, BITS>(a, a.V, a.vn, a.vs, 0, i, h, t0 + j, tid);
      }
      __syncthreads();
      for (int r = wid; r < nr; r += 4) {
        const int t = t0 + lane;
        const bool seen = lane < nt && t < base + (a.kn ? (r0 + r) / a.hq + 1 : 0) && !(t >= plen && t < a.b0[i]);
        float s = -INFINITY;
        if (seen) {
          s = 0.0f;
          for (int c = 0; c < 128; ++c) s = fmaf(sq[r][c], sk[lane][c], s);
          s *= a.scale_log2;
        }
        float m = s;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const float mo = sm[r], mn = fmaxf(mo, m);
        const float ref = mn == -INFINITY ? 0.0f : mn;   // no token so far: every weight below is 0
        const float p = exp2f(s - ref);
        float l = p;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        sp[r][lane] = p;
        __syncwarp();
        if (lane == 0) {
          const float f = exp2f(mo - ref);
          sc[r] = f;
          sm[r] = mn;
          sl[r] = sl[r] * f + l;
        }
      }
      __syncthreads();
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) {
        if (r < nr) {
          float v = acc[r] * sc[r];
          // a key behind the row's own token has weight 0 and must not bring in its value
          const int last = base + (a.kn ? (r0 + r) / a.hq + 1 : 0) - t0;
          for (int j = 0; j < min(nt, last); ++j) v = fmaf(sp[r][j], sv[j][tid], v);
          acc[r] = v;
        }
      }
    }
    __syncthreads();
    const int slot = (int)blockIdx.x - u.tile / a.seg;
#pragma unroll
    for (int r = 0; r < kSimtRows; ++r) {
      if (r < nr) {
        const int64_t qrow = ((int64_t)(a.tok0[i] - a.tok0[0]) + (r0 + r) / a.hq) * a.Hq + h * a.hq + (r0 + r) % a.hq;
        float* p = a.part + (qrow * a.slots + slot) * kPartRow;
        if (tid == 0) p[0] = sm[r], p[1] = sl[r];
        p[4 + tid] = acc[r];
      }
    }
    x = x1;
  }
}

// Query row r of unit (i, h) among the rows of the call.
__device__ __forceinline__ int64_t query_row(const ChunkArgs& a, int i, int h, int r) {
  return ((int64_t)a.tok0[i] + r / a.hq) * a.Hq + h * a.hq + r % a.hq;
}

// One warp: merges the np partial rows of query row qrow, at p0, then p + s * stride (floats),
// and writes the result.
template <typename TO>
__device__ __forceinline__ void combine_row(const ChunkArgs& a, int64_t qrow, const float* p0, const float* p, int stride,
                                            int np) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY;
  for (int s = lane; s < np; s += 32) m = fmaxf(m, *(s == 0 ? p0 : p + (int64_t)s * stride));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int s = 0; s < np; ++s) {
    const float* ps = s == 0 ? p0 : p + (int64_t)s * stride;
    const float2 ml = *reinterpret_cast<const float2*>(ps);
    // a segment without a token that takes part has left no accumulator (a sum of NaN with no maximum: a NaN query)
    const bool some = ml.x != -INFINITY || ml.y != 0.0f;
    const float4 v = some ? reinterpret_cast<const float4*>(ps + 4)[lane] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const float f = some ? exp2f(ml.x - m) : 0.0f;
    l = fmaf(f, some ? ml.y : 0.0f, l);
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);   // no token at all: 0 (NaN stays NaN)
  const int64_t o = qrow * 128 + 4 * lane;
  const float v[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
  if constexpr (sizeof(TO) == 4) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + o) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
    TO w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (std::is_same<TO, __half>::value) w[c] = __float2half_rn(v[c]);
      else w[c] = __float2bfloat16_rn(v[c]);
    }
    *reinterpret_cast<uint2*>(reinterpret_cast<TO*>(a.out) + o) = *reinterpret_cast<uint2*>(w);
  }
}

// One warp per query row of the launch.
template <typename TO>
__global__ void __launch_bounds__(128) chunk_combine(const __grid_constant__ ChunkArgs a, int rows) {
  const int qrow = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (qrow >= rows) return;
  const int t = qrow / a.Hq + a.tok0[0], j = qrow % a.Hq, h = j / a.hq;
  int lo = 0, hi = a.nseq;   // the sequence of token t (empty ones have none)
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.tok0[m] <= t) lo = m;
    else hi = m;
  }
  const int i = lo, r = (t - a.tok0[i]) * a.hq + j % a.hq, blk = r / a.R;
  int before = 0;
  for (int u = lane; u < blk; u += 32) before += a.pad + chunk_unit_tiles(a, i, u);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const int per = (a.tile0[i + 1] - a.tile0[i]) / a.H;
  const int x0 = a.tile0[i] + h * per + before + a.pad, nt = chunk_unit_tiles(a, i, blk);
  const int nseg = nt > 0 ? (x0 + nt - 1) / a.seg - x0 / a.seg + 1 : 0;
  const float* p = a.part + (int64_t)qrow * a.slots * kPartRow;
  combine_row<TO>(a, query_row(a, i, h, r), p, p, kPartRow, nseg * a.par);
}

// Paired row tiles (par = 1) write the rows of units that one CTA covers themselves.
// Here CTA x takes the unit, if any, that run x begins and run x + 1 goes on with.
template <typename TO>
__global__ void __launch_bounds__(256) chunk_join(const __grid_constant__ ChunkArgs a) {
  const int4 p = reinterpret_cast<const int4*>(a.join + blockIdx.x * 8)[0];
  ChunkUnit u;
  u.i = p.x, u.h = p.y, u.t = p.z, u.tile = p.w;
  u.tiles = a.join[blockIdx.x * 8 + 4];
  if (u.tiles == 0) return;
  const int nseg = (u.tile + u.tiles - 1) / a.seg - u.tile / a.seg + 1;
  const int r0 = u.t * a.R, end = min(r0 + a.R, a.n[u.i] * a.hq);
  for (int r = r0 + blockIdx.y * 8 + (threadIdx.x >> 5); r < end; r += gridDim.y * 8) {
    const float* p = a.part + ((int64_t)blockIdx.x * 2 * kRowsUnit + r - r0) * kPartRow;
    combine_row<TO>(a, query_row(a, u.i, u.h, r), p + kRowsUnit * kPartRow, p, 2 * kRowsUnit * kPartRow, nseg);
  }
}

// What a unit costs beside its tiles (its queries, its rows of the result), in tiles. Two
// chunks of 4096 tokens, half of whose units are short, take 525 us at 2, 484 at 4, 467 at 6, 480
// at 8, 493 at 12; 12 ragged chunks of up to 333 tokens 257, 253, 247, 246, 248; 4 rows x 8 tokens
// over 32768 193, 189, 186, 183, 185; 2048 tokens over 8192 430, 427, 428, 431, 436.
constexpr int kUnitPad = 8;

bool chunk_plan(ChunkArgs& a, int num_sms) {
  int ctas = num_sms;
  a.pad = 0;
  if (a.dtype == GEAR_F32) {
    a.R = kSimtRows;
    a.par = 1;
    ctas = 5 * num_sms;   // 38 KB of shared memory each
  } else {
    int most_rows = 0;
    for (int i = 0; i < a.nseq; ++i) most_rows = a.n[i] * a.hq > most_rows ? a.n[i] * a.hq : most_rows;
    // One row tile: both softmax groups on it, alternate tiles. (At 128 rows the two are alike: 8
    // sequences x 32 tokens x 4 query heads over 8192 take 143 us, as half of a pair 141 us.) Up to
    // 32 rows more warps rebuild: 8 x 8 tokens 89 us, else 133 us.
    a.par = most_rows <= 128 ? 2 : 1;
    a.R = a.par == 2 ? 128 : kRowsUnit;
    a.small = most_rows <= 32;
    a.pad = kUnitPad;
  }
  int most = 0;
  int64_t x64 = 0, units_tiles = 0;
  for (int i = 0; i < a.nseq; ++i) {
    a.tile0[i] = (int)x64;
    const int blocks = chunk_blocks(a, i);
    int64_t sum = 0, all = 0;
    for (int t = 0; t < blocks; ++t) {
      const int n = chunk_unit_tiles(a, i, t);
      sum += n > 0 ? a.pad + n : 0;
      if (x64 + sum * a.H > kChunkNumbers) return false;
      all += n;
      most = n > most ? n : most;
    }
    x64 += sum * a.H;
    units_tiles += all * a.H;
  }
  const int x = (int)x64;
  a.tile0[a.nseq] = x;
  a.sms = num_sms;
  // Rebuild tiles ahead where they are read four times or more. 8 sequences over 4096 bf16 tokens x 8
  // heads, rebuilt and fused: two row blocks each 184 and 191 us, three 235 and 270, four 282 and 356,
  // eight 478 and 694; one sequence over 8192 71 and 74, 80 and 89, 91 and 104; 32 fp16 heads over
  // 4096 179 and 178, 230 and 257, 279 and 337. Below four the gain is a seventh at most, for 64 KB
  // of scratch per 96 tokens and head.
  int d = 0;
  for (int i = 0; i < a.nseq; ++i) {
    a.img0[i] = d;
    if (a.n[i] > 0) d += a.H * chunk_unit_tiles(a, i, chunk_blocks(a, i) - 1);
  }
  a.img0[a.nseq] = d;
  if (a.dtype == GEAR_F32 || a.par != 1 || units_tiles < 4 * (int64_t)d) memset(a.img0, 0, sizeof(a.img0));
  a.seg = x > 0 ? (x + ctas - 1) / ctas : 1;
  a.ctas = (x + a.seg - 1) / a.seg;
  a.slots = ((most + a.seg - 1) / a.seg + 1) * a.par;
  return true;
}

static int64_t plan_rows(const ChunkArgs& a) {
  return a.nseq ? (int64_t)(a.tok0[a.nseq - 1] + a.n[a.nseq - 1] - a.tok0[0]) * a.Hq : 0;
}

static size_t part_bytes(const ChunkArgs& a) {
  if (a.dtype != GEAR_F32 && a.par == 1) return (size_t)a.ctas * 2 * kRowsUnit * kPartRow * sizeof(float);
  return ((size_t)plan_rows(a) * a.slots * kPartRow * sizeof(float) + 255) & ~size_t(255);
}

static size_t join_bytes(const ChunkArgs& a) { return ((size_t)a.ctas * 32 + 255) & ~size_t(255); }

size_t chunk_workspace_bytes(const ChunkArgs& a) {
  return part_bytes(a) + join_bytes(a) + (size_t)a.img0[a.nseq] * kImgBytes;
}

static cudaError_t simt_launch(const ChunkArgs& a, cudaStream_t st) {
  switch (a.bits) {
    case 2: chunk_simt<float, 2><<<a.ctas, 128, 0, st>>>(a); break;
    case 4: chunk_simt<float, 4><<<a.ctas, 128, 0, st>>>(a); break;
    default: chunk_simt<float, 8><<<a.ctas, 128, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t chunk_launch(ChunkArgs& a, cudaStream_t st) {
  const int64_t rows = plan_rows(a);
  if (rows == 0) return cudaSuccess;
  uint8_t* ws = reinterpret_cast<uint8_t*>(a.part) + part_bytes(a);
  a.join = reinterpret_cast<int32_t*>(ws);
  a.img = a.img0[a.nseq] > 0 ? ws + join_bytes(a) : nullptr;
  if (a.ctas > 0) {
    const cudaError_t e = a.dtype == GEAR_F32   ? simt_launch(a, st)
                          : a.kc                ? chunk_tc_launch_kc(a, st)
                          : a.dtype == GEAR_F16 ? chunk_tc_launch_f16(a, st)
                                                : chunk_tc_launch_bf16(a, st);
    if (e != cudaSuccess) return e;
  }
  const bool all = a.par == 2 || a.dtype == GEAR_F32;
  if (!all) {   // sequences without a key: nothing has been written
    const size_t row = (size_t)a.Hq * 128 * (a.out_dtype == GEAR_F32 ? 4 : 2);
    for (int i = 0; i < a.nseq; ++i)
      if (a.n[i] > 0 && a.tile0[i + 1] == a.tile0[i]) {
        const cudaError_t e = cudaMemsetAsync(reinterpret_cast<uint8_t*>(a.out) + a.tok0[i] * row, 0, a.n[i] * row, st);
        if (e != cudaSuccess) return e;
      }
    if (a.ctas < 2) return cudaSuccess;
    const dim3 grid(a.ctas - 1, 16);
    if (a.out_dtype == GEAR_F32) chunk_join<float><<<grid, 256, 0, st>>>(a);
    else if (a.out_dtype == GEAR_F16) chunk_join<__half><<<grid, 256, 0, st>>>(a);
    else chunk_join<__nv_bfloat16><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
  }
  const int grid = (int)((rows + 3) / 4);
  if (a.out_dtype == GEAR_F32) chunk_combine<float><<<grid, 128, 0, st>>>(a, (int)rows);
  else if (a.out_dtype == GEAR_F16) chunk_combine<__half><<<grid, 128, 0, st>>>(a, (int)rows);
  else chunk_combine<__nv_bfloat16><<<grid, 128, 0, st>>>(a, (int)rows);
  return cudaGetLastError();
}

}  // namespace gear
