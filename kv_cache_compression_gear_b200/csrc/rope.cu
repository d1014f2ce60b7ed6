// rope.cu -- per-head norm and position rotation of new queries and keys, alone
// (norm_rope) and on the way into the streaming buffers (append_rope).
//
// y = rotate(x * rsqrt(mean_c(x_c^2) + eps) * w) over the 128 channels of a head;
// the rotation takes pairs (a, b) of the first rot_dim channels to
// (a cos - b sin, b cos + a sin), pairs (c, c + rot_dim / 2) or, interleaved,
// (2c, 2c + 1). Everything is binary32, rounded once when y is stored. The
// kernels move two bytes (or four) each way per element and about ten operations:
// memory bound for prompts, launch bound for single tokens. Sixteen lanes hold a
// head, eight consecutive channels each (one 16-byte load of 16-bit values), so
// that the norm is four shuffles and a pair's other half is either in the same
// lane (interleaved) or in the lane rot_dim / 16 away. 8192 tokens of 64 fp16 heads (273 MB)
// take 60 us, 4.5 TB/s or 69 % of the measured copy bandwidth; one token of 40 heads 1.8 us.
#include "common.cuh"
#include "rope.cuh"

namespace gear {

// Warps that fill the device: 148 SMs x 28.
constexpr int64_t kManyWarps = 4096;

template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.v[i];
}

template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&f)[8]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = e[i];
    else if constexpr (std::is_same<T, __half>::value) f[i] = __half2float(e[i]);
    else f[i] = __bfloat162float(e[i]);
  }
}
template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&f)[8]) {
  Raw8<T> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) e[i] = f[i];
    else if constexpr (std::is_same<T, __half>::value) e[i] = __float2half_rn(f[i]);
    else e[i] = __float2bfloat16_rn(f[i]);
  }
  return r;
}

// (cos, sin) of the lane's channels 8l .. 8l + 7: eight pairs when halves are
// paired, four (cs[0 .. 3]) when neighbours are; (1, 0) behind rot_dim.
struct LaneAngles {
  float2 cs[8];
};

__device__ __forceinline__ LaneAngles lane_angles(const RopeSpec& r, int t, int l) {
  LaneAngles a;
#pragma unroll
  for (int i = 0; i < 8; ++i) a.cs[i] = make_float2(1.0f, 0.0f);
  if (!r.table || 8 * l >= r.rot_dim) return a;
  int p = __ldg(r.pos + t);
  if (p < 0 || p >= r.max_pos) {   // reported; the table's edge keeps the read in bounds
    set_device_error(GEAR_ERR_INVALID_ARG);
    p = p < 0 ? 0 : r.max_pos - 1;
  }
  const int half = r.rot_dim / 2;
  const float2* row = r.table + (int64_t)p * half;
  if (r.interleaved) {
    const float4* s = reinterpret_cast<const float4*>(row + 4 * l);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 v = __ldg(s + i);
      a.cs[2 * i] = make_float2(v.x, v.y);
      a.cs[2 * i + 1] = make_float2(v.z, v.w);
    }
  } else {
    const float4* s = reinterpret_cast<const float4*>(row + (8 * l < half ? 8 * l : 8 * l - half));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = __ldg(s + i);
      a.cs[2 * i] = make_float2(v.x, v.y);
      a.cs[2 * i + 1] = make_float2(v.z, v.w);
    }
  }
  return a;
}

// The head held by this half warp, normed (wf: the lane's weights) and rotated; all 16
// lanes take part.
__device__ __forceinline__ void norm_rotate(float (&f)[8], bool norm, const float (&wf)[8], const RopeSpec& r,
                                            const LaneAngles& a, int l) {
  if (norm) {
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s = fmaf(f[i], f[i], s);
      t = fmaf(f[i + 1], f[i + 1], t);
    }
    s += t;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float rs = rsqrtf(s * (1.0f / 128.0f) + r.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f[i] * rs * wf[i];
  }
  if (!r.table) return;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = f[2 * i], y = f[2 * i + 1];
      f[2 * i] = x * a.cs[i].x - y * a.cs[i].y;
      f[2 * i + 1] = y * a.cs[i].x + x * a.cs[i].y;
    }
  } else {
    const int hl = r.rot_dim >> 4;   // lanes of half the rotated channels
    const bool lo = l < hl, in = l < 2 * hl;
    const int src = lo ? l + hl : (in ? l - hl : l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, f[i], src, 16);
      const float v = f[i] * a.cs[i].x + (lo ? -o : o) * a.cs[i].y;
      if (in) f[i] = v;
    }
  }
}

// A warp takes 2 HP heads of one tensor of a token (HP per half warp); grid (tokens / 4,
// groups of heads: those of q, then those of k).
template <typename T, int HP>
__global__ void __launch_bounds__(128) norm_rope(const __grid_constant__ NormRopeArgs a, int qgroups) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), l = threadIdx.x & 15;
  if (t >= a.T) return;
  const bool isq = (int)blockIdx.y < qgroups;
  const HeadView& v = isq ? a.q : a.k;
  const int h0 = ((int)blockIdx.y - (isq ? 0 : qgroups)) * (2 * HP) + ((threadIdx.x >> 4) & 1) * HP;
  const T* src = reinterpret_cast<const T*>(v.x) + t * v.xs + 8 * l;
  Raw8<T> x[HP];
#pragma unroll
  for (int i = 0; i < HP; ++i)   // past the end: the last head again, which is not stored
    x[i] = load8(src + min(h0 + i, v.heads - 1) * 128);
  const LaneAngles ang = lane_angles(a.r, t, l);
  float wf[8];
  if (v.w) unpack8(load8(reinterpret_cast<const T*>(v.w) + 8 * l), wf);
  T* dst = reinterpret_cast<T*>(v.y) + t * v.ys + 8 * l;
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    float f[8];
    unpack8(x[i], f);
    norm_rotate(f, v.w != nullptr, wf, a.r, ang, l);
    if (h0 + i < v.heads) store8(dst + (h0 + i) * 128, pack8<T>(f));
  }
}

// grid (tokens of all entries, chunks of 8 heads): half warp = one head of K and V.
template <typename T>
__global__ void __launch_bounds__(128) append_rope(const __grid_constant__ AppendRopeArgs a) {
  const int ti = blockIdx.x, l = threadIdx.x & 15;
  int lo = 0, hi = a.n;   // entry e with first[e] <= ti < first[e + 1]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.first[m] <= ti) lo = m;
    else hi = m;
  }
  const int e = lo, j = ti - a.first[e];
  const int tau = a.tau0[e] + j;
  const int hw = blockIdx.y * 8 + (threadIdx.x >> 4);
  const int h = min(hw, a.H - 1);   // a half warp past the end repeats the last head and stores nothing
  const int64_t dst = (((int64_t)a.dst[e] * a.H + h) * a.n_b + a.slot0[e] + j) * 128 + 8 * l;
  Raw8<T> kx, vx;
  if (tau < a.fill[e]) {
    const int64_t src = (((int64_t)a.row[e] * a.H + h) * a.n_b + tau) * 128 + 8 * l;
    kx = load8(reinterpret_cast<const T*>(a.kbuf) + src);
    vx = load8(reinterpret_cast<const T*>(a.vbuf) + src);
  } else {
    const int64_t t = a.src0[e] + (tau - a.fill[e]);
    kx = load8(reinterpret_cast<const T*>(a.kn) + t * a.ks + h * 128 + 8 * l);
    vx = load8(reinterpret_cast<const T*>(a.vn) + t * a.vs + h * 128 + 8 * l);
    if (a.w || a.r.table) {
      const LaneAngles ang = lane_angles(a.r, (int)t, l);
      float f[8], wf[8];
      unpack8(kx, f);
      if (a.w) unpack8(load8(reinterpret_cast<const T*>(a.w) + 8 * l), wf);
      norm_rotate(f, a.w != nullptr, wf, a.r, ang, l);
      kx = pack8<T>(f);
    }
  }
  if (hw < a.H) {
    store8(reinterpret_cast<T*>(a.kd) + dst, kx);
    store8(reinterpret_cast<T*>(a.vd) + dst, vx);
  }
  if (a.set && j == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    const int b = a.row[e];
    a.krows[a.B + b] = a.vrows[a.B + b] = a.nblk[e];
    a.krows[2 * a.B + b] = a.vrows[2 * a.B + b] = a.nbuf[e];
  }
}

__global__ void __launch_bounds__(kFillRows) paged_fill(const __grid_constant__ PagedFill a) {
  const int i = threadIdx.x;
  if (i < a.n) a.krows[2 * a.B + a.row[i]] = a.vrows[2 * a.B + a.row[i]] = a.nbuf[i];
}

// Four heads per half warp keep enough loads in flight for prompts; with few heads in
// all, fewer each spread them over more warps: kManyWarps of them for more heads each. Kernel
// times with one, two and four heads per half warp, 64 fp16 heads: 128 tokens (2048 warps of two
// heads each half) 3.5, 3.1, 3.4 us; 256 6.4, 4.6, 4.8; 1024 17, 12.9, 10.5; 8192 120, 80, 60. 40 heads: 16
// tokens 2.2, 2.3, 2.8 us; 512 (2560 warps of four) 6.9, 6.3, 5.2; 1024 11.6, 9.3, 8.4. Four
// also have to leave less than a quarter of the places without a head: 8192 tokens of 3 + 3 heads
// (half of them) 17.9, 12.8, 15.7, of 5 + 1 heads 17.6, 17.5, 15.9.
template <typename T>
static void norm_rope_t(const NormRopeArgs& a, cudaStream_t st) {
  auto groups = [](int heads, int hp) { return (heads + 2 * hp - 1) / (2 * hp); };
  auto warps = [&](int hp) { return (int64_t)a.T * (groups(a.q.heads, hp) + groups(a.k.heads, hp)); };
  auto grid = [&](int hp) { return dim3((a.T + 3) / 4, groups(a.q.heads, hp) + groups(a.k.heads, hp)); };
  if (warps(4) >= kManyWarps && warps(4) * 2 <= warps(2) * 3 / 2) norm_rope<T, 4><<<grid(4), 128, 0, st>>>(a, groups(a.q.heads, 4));
  else if (warps(2) >= kManyWarps) norm_rope<T, 2><<<grid(2), 128, 0, st>>>(a, groups(a.q.heads, 2));
  else norm_rope<T, 1><<<grid(1), 128, 0, st>>>(a, groups(a.q.heads, 1));
}

cudaError_t norm_rope_launch(const NormRopeArgs& a, int dtype, cudaStream_t st) {
  if (a.T == 0 || a.q.heads + a.k.heads == 0) return cudaSuccess;
  if (dtype == GEAR_F32) norm_rope_t<float>(a, st);
  else if (dtype == GEAR_F16) norm_rope_t<__half>(a, st);
  else norm_rope_t<__nv_bfloat16>(a, st);
  return cudaGetLastError();
}

cudaError_t append_rope_launch(const AppendRopeArgs& a, int dtype, cudaStream_t st) {
  if (a.n == 0 || a.first[a.n] == 0) return cudaSuccess;
  const dim3 grid(a.first[a.n], (a.H + 7) / 8);
  if (dtype == GEAR_F32) append_rope<float><<<grid, 128, 0, st>>>(a);
  else if (dtype == GEAR_F16) append_rope<__half><<<grid, 128, 0, st>>>(a);
  else append_rope<__nv_bfloat16><<<grid, 128, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t paged_fill_launch(const PagedFill& a, cudaStream_t st) {
  if (a.n == 0) return cudaSuccess;
  paged_fill<<<1, kFillRows, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace gear
