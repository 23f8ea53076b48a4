// The way from gradients to updated parameters over a list of tensors: the
// global gradient norm with the clipping coefficient, clipping, and Adam with
// decoupled weight decay.  The lists travel as kernel parameters, so a call
// copies nothing to the device first and a captured graph holds its own list.
//
// All three walk the same tiles: tensor k owns tile0[k+1] - tile0[k] tiles of
// kTile values, and block b of G takes the tiles [T b / G, T (b+1) / G) of the
// concatenation, whatever tensors they belong to.  A thread takes 8 values of a
// tile.  Where every array of a tensor allows it, index 0 is moved down to a
// 32-byte (16-bit types: 16-byte) boundary (`shift` values, skipped by the
// first thread), so that views at odd offsets still move as vectors.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <new>

#include "host.h"

namespace spin4d {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                       // values a thread takes of a tile
constexpr int kTile = kThreads * kVec;
constexpr int kMaxBlocks = 1184;              // slots of the norm's partial sums do not depend on the device
constexpr int kNormCap = 1024;                // tensors of one launch; longer lists take several
constexpr int64_t kMaxValues = int64_t(1) << 40;
constexpr int kMaxTensors = 1 << 16;

__host__ __device__ inline int dtype_bytes(int dt) { return dt == SPIN4D_F32 ? 4 : 2; }

// ---------------------------------------------------------------------------
// Lists as the kernels see them
// ---------------------------------------------------------------------------
template <int CAP>
struct NormList {
  int count;
  const void* ptr[CAP];
  int64_t n[CAP];
  uint32_t tile0[CAP + 1];
  uint8_t dtype[CAP];
};

template <int CAP>
struct ClipList {
  int count;
  const void* src[CAP];
  void* dst[CAP];
  int64_t n[CAP];
  uint32_t tile0[CAP + 1];
  uint8_t src_dtype[CAP], dst_dtype[CAP];
  uint8_t shift[CAP];                         // values below index 0 of the aligned tile, or kStrided
};

template <int CAP>
struct AdamList {
  int count;
  float* p[CAP];
  void* work[CAP];
  void* g[CAP];
  float* m[CAP];
  float* v[CAP];
  int64_t n[CAP];
  float lr[CAP], decay[CAP];
  uint32_t tile0[CAP + 1];
  uint8_t g_dtype[CAP], work_dtype[CAP];
  uint8_t shift[CAP];
};
constexpr int kStrided = 255;                 // arrays that are not aligned alike: a warp's lanes take every 32nd value

// Last k with tile0[k] <= tile: the tensor that owns the tile (tensors without values own none).
__device__ __forceinline__ int owner(const uint32_t* tile0, int count, uint32_t tile) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tile0[mid] <= tile) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t block_begin(uint32_t tiles, int b, int blocks) {
  return (uint32_t)((uint64_t)tiles * (uint32_t)b / (uint32_t)blocks);
}
// The block whose range holds the tile: the largest b with block_begin(b) <= tile.
__device__ __forceinline__ int block_of(uint32_t tiles, uint32_t tile, int blocks) {
  return (int)((((uint64_t)tile + 1) * (uint32_t)blocks - 1) / tiles);
}

// ---------------------------------------------------------------------------
// Eight values at once
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
__device__ __forceinline__ void load_vec(const T* a, float x[kVec]);
template <>
__device__ __forceinline__ void load_vec<float>(const float* a, float x[kVec]) {
  const float4 u = reinterpret_cast<const float4*>(a)[0], w = reinterpret_cast<const float4*>(a)[1];
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = w.x; x[5] = w.y; x[6] = w.z; x[7] = w.w;
}
template <>
__device__ __forceinline__ void load_vec<__half>(const __half* a, float x[kVec]) {
  const uint4 u = *reinterpret_cast<const uint4*>(a);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16>(const __nv_bfloat16* a, float x[kVec]) {
  const uint4 u = *reinterpret_cast<const uint4*>(a);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <typename T>
__device__ __forceinline__ void store_vec(T* a, const float x[kVec]);
template <>
__device__ __forceinline__ void store_vec<float>(float* a, const float x[kVec]) {
  reinterpret_cast<float4*>(a)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(a)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
template <>
__device__ __forceinline__ void store_vec<__half>(__half* a, const float x[kVec]) {
  __half2 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(h);
}
template <>
__device__ __forceinline__ void store_vec<__nv_bfloat16>(__nv_bfloat16* a, const float x[kVec]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(a) = *reinterpret_cast<const uint4*>(h);
}

// This thread's 8 places of one tile of a tensor of n values: first + i * stride for i in [0, 8),
// those in [0, n).  `whole`: all of them are, and they are neighbours on a vector's boundary.
struct Places {
  int64_t first;
  int stride;
  bool whole;
};
__device__ __forceinline__ Places places(uint32_t tile_in_tensor, int shift, int64_t n) {
  Places q;
  const int64_t base = (int64_t)tile_in_tensor * kTile;
  if (shift == kStrided) {
    q.first = base + (threadIdx.x >> 5) * (32 * kVec) + (threadIdx.x & 31);
    q.stride = 32;
    q.whole = false;
  } else {
    q.first = base + threadIdx.x * kVec - shift;
    q.stride = 1;
    q.whole = q.first >= 0 && q.first + kVec <= n;
  }
  return q;
}

template <typename T>
__device__ __forceinline__ void load8(const T* a, const Places& q, int64_t n, float x[kVec]) {
  if (q.whole) {
    load_vec<T>(a + q.first, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t j = q.first + (int64_t)i * q.stride;
    x[i] = j >= 0 && j < n ? to_f<T>(a[j]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* a, const Places& q, int64_t n, const float x[kVec]) {
  if (q.whole) {
    store_vec<T>(a + q.first, x);
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int64_t j = q.first + (int64_t)i * q.stride;
    if (j >= 0 && j < n) a[j] = from_f<T>(x[i]);
  }
}
__device__ __forceinline__ void load8(const void* a, int dt, const Places& q, int64_t n, float x[kVec]) {
  if (dt == SPIN4D_F32) load8(static_cast<const float*>(a), q, n, x);
  else if (dt == SPIN4D_F16) load8(static_cast<const __half*>(a), q, n, x);
  else load8(static_cast<const __nv_bfloat16*>(a), q, n, x);
}
__device__ __forceinline__ void store8(void* a, int dt, const Places& q, int64_t n, const float x[kVec]) {
  if (dt == SPIN4D_F32) store8(static_cast<float*>(a), q, n, x);
  else if (dt == SPIN4D_F16) store8(static_cast<__half*>(a), q, n, x);
  else store8(static_cast<__nv_bfloat16*>(a), q, n, x);
}

// ---------------------------------------------------------------------------
// Norm.  Squares and sums are 64-bit: a square of any fp32 value and the sum
// of 2^40 of them neither overflow nor vanish, and the sum's order does not
// show in the 32-bit result.  No atomics: block b's part of tensor k goes to
// slot b + k (along the walk over (b, k) one of the two grows at each part, so
// no two parts share a slot), and one block adds the slots in a fixed order.
// ---------------------------------------------------------------------------
enum { kL1 = SPIN4D_NORM_L1, kL2 = SPIN4D_NORM_L2, kMax = SPIN4D_NORM_MAX };

template <int NORM>
__device__ __forceinline__ double join(double a, double b) {
  if (NORM == kMax) return (a > b || isnan(a)) ? a : b;   // a NaN stays
  return a + b;
}
template <int NORM>
__device__ __forceinline__ void take(double& acc, const float x[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const double d = (double)x[i];
    if (NORM == kL2) acc = fma(d, d, acc);
    else acc = join<NORM>(acc, fabs(d));
  }
}
template <int NORM>
__device__ __forceinline__ double warp_join(double a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = join<NORM>(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

template <int CAP, int NORM>
__global__ void __launch_bounds__(kThreads) norm_parts_kernel(const __grid_constant__ NormList<CAP> list,
                                                              double* __restrict__ slots) {
  __shared__ double part[kThreads / 32];
  const uint32_t tiles = list.tile0[list.count];
  uint32_t t = block_begin(tiles, blockIdx.x, gridDim.x);
  const uint32_t end = block_begin(tiles, blockIdx.x + 1, gridDim.x);
  if (t >= end) return;
  for (int k = owner(list.tile0, list.count, t); t < end; ++k) {
    const uint32_t stop = min(end, list.tile0[k + 1]);
    if (t >= stop) continue;                  // a tensor without values
    const int dt = list.dtype[k], bytes = dtype_bytes(dt);
    const int64_t n = list.n[k];
    const int shift = (int)((reinterpret_cast<uintptr_t>(list.ptr[k]) & (kVec * bytes - 1)) / bytes);
    double acc = 0.0;
    for (; t < stop; ++t) {
      const Places q = places(t - list.tile0[k], shift, n);
      float x[kVec];
      load8(list.ptr[k], dt, q, n, x);
      take<NORM>(acc, x);
    }
    acc = warp_join<NORM>(acc);
    __syncthreads();                          // the last tensor's parts have been read
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kThreads / 32; ++w) acc = join<NORM>(acc, part[w]);
      slots[blockIdx.x + k] = acc;
    }
  }
}

struct FinishArgs {
  double grad_scale, max_norm;
  int blocks, first, last;
  spin4d_grad_control* control;
  float* norms;                               // this launch's tensors' (may be null)
  double* total;                              // carried from launch to launch of one list
  const double* slots;
};

template <int CAP, int NORM>
__global__ void __launch_bounds__(1024) norm_finish_kernel(const __grid_constant__ NormList<CAP> list,
                                                           const FinishArgs f) {
  __shared__ double part[32];
  const uint32_t tiles = list.tile0[list.count];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double mine = 0.0;
  for (int k = warp; k < list.count; k += 32) {
    const uint32_t a = list.tile0[k], e = list.tile0[k + 1];
    double s = 0.0;
    if (e > a) {
      const int lb = block_of(tiles, e - 1, f.blocks);
      for (int b = block_of(tiles, a, f.blocks) + lane; b <= lb; b += 32) s = join<NORM>(s, f.slots[b + k]);
    }
    s = warp_join<NORM>(s);
    if (lane == 0 && f.norms) f.norms[k] = (float)(f.grad_scale * (NORM == kL2 ? sqrt(s) : s));
    mine = join<NORM>(mine, s);
  }
  if (lane == 0) part[warp] = mine;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double total = f.first ? 0.0 : *f.total;
  for (int w = 0; w < 32; ++w) total = join<NORM>(total, part[w]);
  *f.total = total;
  if (!f.last) return;
  const double norm = f.grad_scale * (NORM == kL2 ? sqrt(total) : total);
  const float norm32 = (float)norm;
  const bool fine = isfinite(norm32);
  f.control->norm = norm32;
  f.control->coef = fine ? (float)(f.grad_scale * fmin(1.0, f.max_norm / (norm + 1e-6))) : 0.0f;
  if (fine) f.control->step += 1;
  else f.control->skipped += 1;
}

// ---------------------------------------------------------------------------
// Clip: out = coef * gradient.
// ---------------------------------------------------------------------------
template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ ClipList<CAP> list,
                                                        const spin4d_grad_control* __restrict__ control) {
  const uint32_t tiles = list.tile0[list.count];
  uint32_t t = block_begin(tiles, blockIdx.x, gridDim.x);
  const uint32_t end = block_begin(tiles, blockIdx.x + 1, gridDim.x);
  if (t >= end) return;
  const float coef = control->coef;
  for (int k = owner(list.tile0, list.count, t); t < end; ++k) {
    const uint32_t stop = min(end, list.tile0[k + 1]);
    for (; t < stop; ++t) {
      const int64_t n = list.n[k];
      const Places q = places(t - list.tile0[k], list.shift[k], n);
      float x[kVec];
      load8(list.src[k], list.src_dtype[k], q, n, x);
#pragma unroll
      for (int i = 0; i < kVec; ++i) x[i] = coef == 0.0f ? 0.0f : coef * x[i];   // zeros whatever the gradient holds
      store8(list.dst[k], list.dst_dtype[k], q, n, x);
    }
  }
}

// ---------------------------------------------------------------------------
// Adam with decoupled weight decay.
// ---------------------------------------------------------------------------
struct AdamArgs {
  float b1, b2, omb1, omb2, eps;
  double log_b1, log_b2;                      // for a step that only the device knows
  int step;                                   // 0: the control's
  int zero_grad;
  const spin4d_grad_control* control;         // may be null
  int32_t* flag;                              // may be null
};

template <int CAP>
__global__ void __launch_bounds__(kThreads) adam_list_kernel(const __grid_constant__ AdamList<CAP> list,
                                                             const AdamArgs a) {
  const uint32_t tiles = list.tile0[list.count];
  uint32_t t = block_begin(tiles, blockIdx.x, gridDim.x);
  const uint32_t end = block_begin(tiles, blockIdx.x + 1, gridDim.x);
  if (t >= end) return;
  float coef = 1.0f;
  int step = a.step;
  bool skip = false;
  if (a.control) {
    coef = a.control->coef;
    if (step == 0) step = a.control->step;
    skip = !isfinite(a.control->norm) || step < 1;
  }
  if (skip && !a.zero_grad) return;
  // 1 - b^step = -expm1(step log b): the product in 64 bits, then within 2 ulp of fp32
  const float inv_bc1 = 1.0f / -expm1f((float)(step * a.log_b1));
  const float inv_bc2 = 1.0f / -expm1f((float)(step * a.log_b2));
  bool bad = false;
  for (int k = owner(list.tile0, list.count, t); t < end; ++k) {
    const uint32_t stop = min(end, list.tile0[k + 1]);
    for (; t < stop; ++t) {
      const int64_t n = list.n[k];
      const Places q = places(t - list.tile0[k], list.shift[k], n);
      if (!skip) {
        const float lr = list.lr[k], decay = lr * list.decay[k];
        float g[kVec], p[kVec], m[kVec], v[kVec];
        load8(list.g[k], list.g_dtype[k], q, n, g);
        load8(list.p[k], q, n, p);
        load8(list.m[k], q, n, m);
        load8(list.v[k], q, n, v);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float gi = coef == 0.0f ? 0.0f : coef * g[i];
          m[i] = a.b1 * m[i] + a.omb1 * gi;
          v[i] = a.b2 * v[i] + a.omb2 * (gi * gi);
          const float mh = m[i] * inv_bc1, vh = v[i] * inv_bc2;
          // outside [0, n) all four are 0: with eps = 0 the quotient is NaN there, which neither is stored nor flagged
          const float r = p[i] - (lr * mh / (sqrtf(vh) + a.eps) + decay * p[i]);
          const int64_t j = q.first + (int64_t)i * q.stride;
          bad |= !isfinite(r) && (q.whole || (j >= 0 && j < n));
          p[i] = r;
        }
        store8(list.p[k], q, n, p);
        store8(list.m[k], q, n, m);
        store8(list.v[k], q, n, v);
        if (list.work[k]) store8(list.work[k], list.work_dtype[k], q, n, p);
      }
      if (a.zero_grad) {
        const float zero[kVec] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        store8(list.g[k], list.g_dtype[k], q, n, zero);
      }
    }
  }
  if (a.flag && __syncthreads_or(bad) && threadIdx.x == 0) atomicExch(a.flag, 1);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool dtype_ok(int dt) { return dt == SPIN4D_F32 || dt == SPIN4D_F16 || dt == SPIN4D_BF16; }

bool array_ok(const void* p, int64_t n, int bytes) { return n == 0 || (p && aligned(p, bytes)); }

// A stretch of memory that a call reads or writes.
struct Stretch {
  uintptr_t lo, hi;
  bool write;
};

// Stretches, on the stack for short lists.  `ok` is false when the host has no memory for a long one.
struct Stretches {
  static constexpr int kLocal = 320;
  Stretch local[kLocal];
  Stretch* at;
  int count = 0;
  explicit Stretches(int most) : at(most <= kLocal ? local : new (std::nothrow) Stretch[most]) {}
  ~Stretches() {
    if (at != local) delete[] at;
  }
  Stretches(const Stretches&) = delete;
  Stretches& operator=(const Stretches&) = delete;
  bool ok() const { return at != nullptr; }
  void add(const void* p, int64_t n, int bytes, bool write) {
    if (p && n > 0) at[count++] = {(uintptr_t)p, (uintptr_t)p + (uint64_t)n * bytes, write};
  }
  // Whether something written is also another array's: blocks run in no order, so the result would have none.
  bool clash() {
    std::sort(at, at + count, [](const Stretch& a, const Stretch& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (int i = 0; i < count; ++i) {
      if (at[i].lo < (at[i].write ? any : written)) return true;
      any = std::max(any, at[i].hi);
      if (at[i].write) written = std::max(written, at[i].hi);
    }
    return false;
  }
};

int shift_of(const void* p, int bytes) { return (int)(((uintptr_t)p & (kVec * bytes - 1)) / bytes); }

// Appends a tensor's tiles; false when the list holds more than a launch can number.
bool add_tiles(uint32_t* tile0, int k, int64_t n, int shift) {
  const int64_t tiles = n == 0 ? 0 : (n + shift + kTile - 1) / kTile;
  const int64_t sum = (int64_t)tile0[k] + tiles;
  tile0[k + 1] = (uint32_t)sum;
  return sum < (int64_t(1) << 31);
}

int blocks_for(uint32_t tiles) { return std::min(persistent_blocks(tiles, 8), kMaxBlocks); }

template <int CAP, int NORM>
int norm_launches(const spin4d_grad_tensor* ts, int count, FinishArgs f, double* slots, cudaStream_t s) {
  float* norms = f.norms;
  int at = 0;
  do {
    NormList<CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_grad_tensor& t = ts[at + k];
      list.ptr[k] = t.grad;
      list.n[k] = t.n;
      list.dtype[k] = (uint8_t)t.grad_dtype;
      if (!add_tiles(list.tile0, k, t.n, shift_of(t.grad, dtype_bytes(t.grad_dtype)))) return SPIN4D_ERR_INVALID;
    }
    const uint32_t tiles = list.tile0[list.count];
    f.blocks = blocks_for(tiles);
    f.first = at == 0;
    f.last = at + list.count == count;
    f.norms = norms ? norms + at : nullptr;
    if (tiles) {
      norm_parts_kernel<CAP, NORM><<<f.blocks, kThreads, 0, s>>>(list, slots);
      SPIN4D_CHECK(launch_status());
    }
    norm_finish_kernel<CAP, NORM><<<1, 1024, 0, s>>>(list, f);
    SPIN4D_CHECK(launch_status());
    at += list.count;
  } while (at < count);
  return SPIN4D_OK;
}

template <int NORM>
int norm_list(const spin4d_grad_tensor* ts, int count, const FinishArgs& f, double* slots, cudaStream_t s) {
  if (count <= 16) return norm_launches<16, NORM>(ts, count, f, slots, s);
  return norm_launches<kNormCap, NORM>(ts, count, f, slots, s);
}

template <int CAP>
int clip_launches(const spin4d_grad_tensor* ts, int count, const spin4d_grad_control* control, cudaStream_t s) {
  for (int at = 0; at < count; at += CAP) {
    ClipList<CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_grad_tensor& t = ts[at + k];
      list.src[k] = t.grad;
      list.dst[k] = t.out ? t.out : const_cast<void*>(t.grad);
      list.n[k] = t.n;
      list.src_dtype[k] = (uint8_t)t.grad_dtype;
      list.dst_dtype[k] = (uint8_t)(t.out ? t.out_dtype : t.grad_dtype);
      int shift = shift_of(t.grad, dtype_bytes(t.grad_dtype));
      if (shift != shift_of(list.dst[k], dtype_bytes(list.dst_dtype[k]))) shift = kStrided;
      list.shift[k] = (uint8_t)shift;
      if (!add_tiles(list.tile0, k, t.n, shift == kStrided ? 0 : shift)) return SPIN4D_ERR_INVALID;
    }
    const uint32_t tiles = list.tile0[list.count];
    if (!tiles) continue;
    clip_kernel<CAP><<<blocks_for(tiles), kThreads, 0, s>>>(list, control);
    SPIN4D_CHECK(launch_status());
  }
  return SPIN4D_OK;
}

template <int CAP>
int adam_launches(const spin4d_adam_tensor* ts, int count, const AdamArgs& a, cudaStream_t s) {
  for (int at = 0; at < count; at += CAP) {
    AdamList<CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_adam_tensor& t = ts[at + k];
      list.p[k] = t.params;
      list.work[k] = t.params_work;
      list.g[k] = t.grad;
      list.m[k] = t.m;
      list.v[k] = t.v;
      list.n[k] = t.n;
      list.lr[k] = t.lr;
      list.decay[k] = t.weight_decay;
      list.g_dtype[k] = (uint8_t)t.grad_dtype;
      list.work_dtype[k] = (uint8_t)t.work_dtype;
      int shift = shift_of(t.params, 4);
      if (shift != shift_of(t.grad, dtype_bytes(t.grad_dtype)) || shift != shift_of(t.m, 4) ||
          shift != shift_of(t.v, 4) || (t.params_work && shift != shift_of(t.params_work, 2)))
        shift = kStrided;
      list.shift[k] = (uint8_t)shift;
      if (!add_tiles(list.tile0, k, t.n, shift == kStrided ? 0 : shift)) return SPIN4D_ERR_INVALID;
    }
    const uint32_t tiles = list.tile0[list.count];
    if (!tiles) continue;
    adam_list_kernel<CAP><<<blocks_for(tiles), kThreads, 0, s>>>(list, a);
    SPIN4D_CHECK(launch_status());
  }
  return SPIN4D_OK;
}

}  // namespace
}  // namespace spin4d

using namespace spin4d;

extern "C" size_t spin4d_grad_norm_workspace(int count) {
  if (count < 0 || count > kMaxTensors) return 0;
  return sizeof(double) * (1 + kMaxBlocks + kNormCap);
}

extern "C" int spin4d_grad_norm(const spin4d_grad_tensor* tensors, int count, int norm_type, double grad_scale,
                                double max_norm, spin4d_grad_control* control, float* norms, void* workspace,
                                size_t ws_bytes, spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (norm_type != kL1 && norm_type != kL2 && norm_type != kMax) return SPIN4D_ERR_INVALID;
  if (!(grad_scale > 0.0) || !isfinite(grad_scale) || !(max_norm >= 0.0)) return SPIN4D_ERR_INVALID;
  if (!control || !aligned(control, 16) || (norms && !aligned(norms, 4))) return SPIN4D_ERR_INVALID;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < spin4d_grad_norm_workspace(count)) return SPIN4D_ERR_INVALID;
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    const spin4d_grad_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxValues || !dtype_ok(t.grad_dtype)) return SPIN4D_ERR_INVALID;
    if (!array_ok(t.grad, t.n, dtype_bytes(t.grad_dtype))) return SPIN4D_ERR_INVALID;
    tiles += t.n / kTile + 2;
  }
  if (tiles >= (int64_t(1) << 31)) return SPIN4D_ERR_INVALID;
  if (fault_injected("spin4d_grad_norm")) return SPIN4D_ERR_INJECTED;
  FinishArgs f = {};
  f.grad_scale = grad_scale;
  f.max_norm = max_norm;
  f.control = control;
  f.norms = norms;
  f.total = static_cast<double*>(workspace);
  double* slots = static_cast<double*>(workspace) + 1;
  f.slots = slots;
  const cudaStream_t s = (cudaStream_t)stream;
  if (norm_type == kL2) return norm_list<kL2>(tensors, count, f, slots, s);
  if (norm_type == kL1) return norm_list<kL1>(tensors, count, f, slots, s);
  return norm_list<kMax>(tensors, count, f, slots, s);
}

extern "C" int spin4d_clip_grads(const spin4d_grad_tensor* tensors, int count, const spin4d_grad_control* control,
                                 spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (!control || !aligned(control, 16)) return SPIN4D_ERR_INVALID;
  Stretches used(2 * count);
  if (!used.ok()) return SPIN4D_ERR_INVALID;
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    const spin4d_grad_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxValues || !dtype_ok(t.grad_dtype) || (t.out && !dtype_ok(t.out_dtype)))
      return SPIN4D_ERR_INVALID;
    if (!array_ok(t.grad, t.n, dtype_bytes(t.grad_dtype))) return SPIN4D_ERR_INVALID;
    if (t.out && !array_ok(t.out, t.n, dtype_bytes(t.out_dtype))) return SPIN4D_ERR_INVALID;
    if (!t.out || (t.out == t.grad && t.out_dtype == t.grad_dtype)) {
      used.add(t.grad, t.n, dtype_bytes(t.grad_dtype), true);
    } else {
      used.add(t.grad, t.n, dtype_bytes(t.grad_dtype), false);
      used.add(t.out, t.n, dtype_bytes(t.out_dtype), true);
    }
    tiles += t.n / kTile + 2;
  }
  if (tiles >= (int64_t(1) << 31) || used.clash()) return SPIN4D_ERR_INVALID;
  if (fault_injected("spin4d_clip_grads")) return SPIN4D_ERR_INJECTED;
  if (count <= 16) return clip_launches<16>(tensors, count, control, (cudaStream_t)stream);
  return clip_launches<1024>(tensors, count, control, (cudaStream_t)stream);
}

extern "C" int spin4d_adam_step_tensors(const spin4d_adam_tensor* tensors, int count, int step, double b1, double b2,
                                        double eps, int zero_grad, const spin4d_grad_control* control,
                                        int32_t* nonfinite_flag, spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (step < 0 || (step == 0 && !control)) return SPIN4D_ERR_INVALID;
  // as the kernel holds them: a rate that rounds to 1 would never forget
  if (!(b1 >= 0.0 && (float)b1 < 1.0f && b2 >= 0.0 && (float)b2 < 1.0f && eps >= 0.0 && isfinite((float)eps)))
    return SPIN4D_ERR_INVALID;
  if ((control && !aligned(control, 16)) || (nonfinite_flag && !aligned(nonfinite_flag, 4))) return SPIN4D_ERR_INVALID;
  Stretches used(5 * count);
  if (!used.ok()) return SPIN4D_ERR_INVALID;
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    const spin4d_adam_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxValues || !isfinite(t.lr) || !isfinite(t.weight_decay)) return SPIN4D_ERR_INVALID;
    if (!dtype_ok(t.grad_dtype)) return SPIN4D_ERR_INVALID;
    if (t.params_work && ((t.work_dtype != SPIN4D_F16 && t.work_dtype != SPIN4D_BF16) || !aligned(t.params_work, 2)))
      return SPIN4D_ERR_INVALID;
    if (!array_ok(t.params, t.n, 4) || !array_ok(t.m, t.n, 4) || !array_ok(t.v, t.n, 4) ||
        !array_ok(t.grad, t.n, dtype_bytes(t.grad_dtype)))
      return SPIN4D_ERR_INVALID;
    used.add(t.params, t.n, 4, true);
    used.add(t.m, t.n, 4, true);
    used.add(t.v, t.n, 4, true);
    used.add(t.params_work, t.n, 2, true);
    used.add(t.grad, t.n, dtype_bytes(t.grad_dtype), zero_grad != 0);
    tiles += t.n / kTile + 2;
  }
  if (tiles >= (int64_t(1) << 31) || used.clash()) return SPIN4D_ERR_INVALID;
  if (fault_injected("spin4d_adam_step_tensors")) return SPIN4D_ERR_INJECTED;
  AdamArgs a;
  a.b1 = (float)b1;
  a.b2 = (float)b2;
  a.omb1 = (float)(1.0 - b1);
  a.omb2 = (float)(1.0 - b2);
  a.eps = (float)eps;
  a.log_b1 = log(b1);
  a.log_b2 = log(b2);
  a.step = step;
  a.zero_grad = zero_grad ? 1 : 0;
  a.control = control;
  a.flag = nonfinite_flag;
  if (count <= 16) return adam_launches<16>(tensors, count, a, (cudaStream_t)stream);
  return adam_launches<512>(tensors, count, a, (cudaStream_t)stream);
}
