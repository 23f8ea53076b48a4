// The way from gradients to updated parameters over a list of tensors: the
// global gradient norm with the clipping coefficient, clipping, and Adam with
// decoupled weight decay.  The lists travel as kernel parameters, so a call
// copies nothing to the device first and a captured graph holds its own list.
//
// All three walk the same tiles: tensor k owns tile0[k+1] - tile0[k] tiles of
// kTile values, and block b takes the tiles [per b, per (b+1)) of the
// concatenation, whatever tensors they belong to.  A thread takes 8 values of a
// tile.  Where every array of a tensor allows it, index 0 is moved down to a
// 32-byte (16-bit types: 16-byte) boundary (`shift` values, skipped by the
// first thread), so that views at odd offsets still move as vectors.
//
// The norm reads upwards, clip and Adam downwards: what the norm read last is
// what the L2 still holds.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <new>

#include "host.h"
#include "pdl.cuh"

namespace spin4d {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 8;                       // values a thread takes of a tile
constexpr int kTile = kThreads * kVec;
constexpr int kMaxNormBlocks = 480;           // the norm's workspace does not depend on the device
constexpr int kNormCap = 1024;                // tensors of one launch; longer lists take several
constexpr int64_t kMaxValues = int64_t(1) << 40;
constexpr int kMaxTensors = 1 << 16;

// Blocks of a launch, at most, for each SM.  The norm's are all resident at once, each writes slots that one block
// adds in the end: with 2, 3, 4 and 5 a SM the norm of 134M fp16 values takes 49.3, 44.8, 46.8 and 46.7 us, of 300
// small tensors 8.0, 7.2, 8.6 and 10.8.  Clip and Adam meet nowhere: short blocks that the hardware hands
// out as others end keep loads and stores mixed and both dies busy.  Adam over 134M parameters: 669 us with 3
// a SM (all resident), 618 with 32, 602 with 64, 595 with 128; norm and clip of 16.8M fp16 values into fp32:
// 36.0 us with 4, 27.5 with 8, 26.4 with 32, 30.8 with 64; of 11.5M fp32: 25.5, 25.0, 23.6 and 23.1.
constexpr int kNormBlocks = 3, kClipBlocks = 32, kAdamBlocks = 96;
// Tiles that a tensor of a long list counts for besides its own (see norm_launches).
constexpr uint32_t kTensorTiles = 6;

__host__ __device__ inline int dtype_bytes(int dt) { return dt == SPIN4D_F32 ? 4 : 2; }

// What the checked build verifies on the device (a failure is recorded and the access left out or made value by value);
// elsewhere it holds and costs nothing.
__device__ __forceinline__ bool expect(bool ok) {
#ifdef SPIN4D_CHECKED
  return bounds_ok(ok);
#else
  return true;
#endif
}

// ---------------------------------------------------------------------------
// Lists as the kernels see them
// ---------------------------------------------------------------------------
// A tensor's length, types and the values that lie below index 0 in its first tile, in one word.
constexpr int kStrided = 15;                  // instead of a shift: written arrays that are not aligned alike
struct Meta {
  uint64_t bits;
  __host__ __device__ int64_t n() const { return (int64_t)(bits & ((uint64_t(1) << 48) - 1)); }
  __host__ __device__ int dtype() const { return (int)(bits >> 48) & 15; }
  __host__ __device__ int out_dtype() const { return (int)(bits >> 52) & 15; }
  __host__ __device__ int shift() const { return (int)(bits >> 56) & 15; }
  // a gradient that is only read, and not aligned like what is written
  __host__ __device__ bool loose() const { return (bits >> 60) & 1; }
};
Meta meta_of(int64_t n, int dtype, int out_dtype, int shift, bool loose) {
  return {(uint64_t)n | (uint64_t)dtype << 48 | (uint64_t)out_dtype << 52 | (uint64_t)shift << 56 | (uint64_t)loose << 60};
}

// What a kernel reads of one tensor lies together: each line of the constant bank that a block touches
// for the first time costs it a round trip.
struct NormEntry {
  const void* a;
  Meta meta;
};
struct ClipEntry {
  const void* a;
  void* out;
  Meta meta;
};
struct alignas(64) AdamEntry {
  float* p;
  float* m;
  float* v;
  void* g;
  void* work;
  Meta meta;
  float lr, decay;
};

constexpr int kHints = 128;
template <typename Entry, int CAP>
struct List {
  int count;
  uint32_t tiles;
  uint32_t per;                               // tiles of a block
  uint32_t hint_shift;
  uint32_t tile0[CAP + 1];
  uint16_t hint[CAP > 16 ? kHints + 1 : 2];   // the owner of each 2^hint_shift-th tile, and the last tensor
  Entry at[CAP];

  // The last tensor that begins at or before the tile: its owner (tensors without values own none).
  __device__ __forceinline__ int owner(uint32_t tile) const {
    const int k = find(tile);
    expect(tile >= tiles || (tile0[k] <= tile && tile < tile0[k + 1]));
    return k;
  }
  __device__ __forceinline__ int find(uint32_t tile) const {
    if (CAP <= 16) {
      int k = 0;
      while (k + 1 < count && tile0[k + 1] <= tile) ++k;
      return k;
    }
    int lo = hint[tile >> hint_shift], hi = hint[(tile >> hint_shift) + 1] + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile0[mid] <= tile) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};

// ---------------------------------------------------------------------------
// Eight values at once
// ---------------------------------------------------------------------------
// kStream: the line's next use is far off, so it is the first to leave L2.  32-byte accesses say so; a 16-byte
// load that skips L1 does it too (an fp16 gradient read that way by the norm was gone when clip came: 34.0 us
// for both over 16.8M values, 31.2 read plainly).
enum Hint { kKeep, kStream };

// 8 values of 4 or 2 bytes as they are in memory.
template <int BYTES>
struct Raw {
  uint32_t w[kVec * BYTES / 4];
};
template <Hint H>
__device__ __forceinline__ void load_raw(const void* a, Raw<4>& r) {
  if (H == kStream)
    asm volatile("ld.global.L1::no_allocate.L2::evict_first.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(a) : "memory");
  else
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                   "=r"(r.w[7])
                 : "l"(a) : "memory");
}
template <Hint H>
__device__ __forceinline__ void load_raw(const void* a, Raw<2>& r) {
  if (H == kStream)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(a) : "memory");
  else
    asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(a) : "memory");
}
__device__ __forceinline__ void store_raw(void* a, const Raw<4>& r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(a), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]),
               "r"(r.w[3]), "r"(r.w[4]), "r"(r.w[5]), "r"(r.w[6]), "r"(r.w[7])
               : "memory");
}
__device__ __forceinline__ void store_raw(void* a, const Raw<2>& r) {
  asm volatile("st.global.v4.b32 [%0], {%1,%2,%3,%4};" ::"l"(a), "r"(r.w[0]), "r"(r.w[1]), "r"(r.w[2]), "r"(r.w[3])
               : "memory");
}

// `bf`: 16-bit values are bfloat16, else fp16.
__device__ __forceinline__ void unpack(const Raw<4>& r, bool, float x[kVec]) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) x[i] = __uint_as_float(r.w[i]);
}
__device__ __forceinline__ void unpack(const Raw<2>& r, bool bf, float x[kVec]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    x[2 * i] = bf ? __uint_as_float(r.w[i] << 16) : f.x;
    x[2 * i + 1] = bf ? __uint_as_float(r.w[i] & 0xffff0000u) : f.y;
  }
}
__device__ __forceinline__ void pack(const float x[kVec], bool, Raw<4>& r) {
#pragma unroll
  for (int i = 0; i < kVec; ++i) r.w[i] = __float_as_uint(x[i]);
}
__device__ __forceinline__ void pack(const float x[kVec], bool bf, Raw<2>& r) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    r.w[i] = bf ? *reinterpret_cast<const uint32_t*>(&b) : *reinterpret_cast<const uint32_t*>(&h);
  }
}

// This thread's 8 places of one tile of a tensor of n values: first + i * stride for i in [0, 8),
// those in [0, n).  `whole`: all of them are, and they are neighbours on a vector's boundary.
struct Places {
  int64_t first, n;
  int stride;
  bool whole;
  __device__ __forceinline__ Places(uint32_t tile, int shift, int64_t n_) : n(n_) {
    const int64_t base = (int64_t)tile * kTile;
    if (shift == kStrided) {
      first = base + (threadIdx.x >> 5) * (32 * kVec) + (threadIdx.x & 31);
      stride = 32;
      whole = false;
    } else {
      first = base + threadIdx.x * kVec - shift;
      stride = 1;
      whole = first >= 0 && first + kVec <= n;
    }
  }
  // whole places are one vector of an array that is aligned with them
  __device__ __forceinline__ bool vector_in(const void* a, int bytes) const {
    return ((uintptr_t)a + first * bytes) % (kVec * bytes) == 0;
  }
  __device__ __forceinline__ int64_t place(int i) const { return first + (int64_t)i * stride; }
  __device__ __forceinline__ bool has(int i) const { return place(i) >= 0 && place(i) < n; }
};

// Into L2 ahead of the loads: a launch that overlaps the kernel before it may not read yet, but may ask.
__device__ __forceinline__ void warm(const void* a, const Places& q, int bytes) {
  if (q.whole) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a) + q.first * bytes));
}

// The values at the places; 0 for those outside [0, n).  `loose`: the array is not aligned with the places; a
// thread's neighbouring values then come one by one, the later ones out of L1.  (Norm and update of 16.8M with
// bf16 gradients an odd value into their buffer: 79.8 us, aligned 77.9, every array a value at a time 90.7.)
template <Hint H>
__device__ __forceinline__ void fetch(const void* a, const Places& q, Raw<4>& r, bool loose = false) {
  if (q.whole && !loose && expect(q.vector_in(a, 4))) {
    load_raw<H>(static_cast<const float*>(a) + q.first, r);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) r.w[i] = q.has(i) ? static_cast<const uint32_t*>(a)[q.place(i)] : 0u;
  }
}
template <Hint H>
__device__ __forceinline__ void fetch(const void* a, const Places& q, Raw<2>& r, bool loose = false) {
  if (q.whole && !loose && expect(q.vector_in(a, 2))) {
    load_raw<H>(static_cast<const uint16_t*>(a) + q.first, r);
  } else {
    uint32_t h[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) h[i] = q.has(i) ? static_cast<const uint16_t*>(a)[q.place(i)] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = h[2 * i] | h[2 * i + 1] << 16;
  }
}
__device__ __forceinline__ void put(void* a, const Places& q, const Raw<4>& r) {
  if (q.whole && expect(q.vector_in(a, 4))) {
    store_raw(static_cast<float*>(a) + q.first, r);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (q.has(i)) static_cast<uint32_t*>(a)[q.place(i)] = r.w[i];
  }
}
__device__ __forceinline__ void put(void* a, const Places& q, const Raw<2>& r) {
  if (q.whole && expect(q.vector_in(a, 2))) {
    store_raw(static_cast<uint16_t*>(a) + q.first, r);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (q.has(i)) static_cast<uint16_t*>(a)[q.place(i)] = (uint16_t)(r.w[i / 2] >> 16 * (i & 1));
  }
}
__device__ __forceinline__ void put(void* a, int dt, const Places& q, const float x[kVec]) {
  if (dt == SPIN4D_F32) {
    Raw<4> r;
    pack(x, false, r);
    put(a, q, r);
  } else {
    Raw<2> r;
    pack(x, dt == SPIN4D_BF16, r);
    put(a, q, r);
  }
}

// ---------------------------------------------------------------------------
// Norm.  Squares and sums are 64-bit: a square of any fp32 value and the sum
// of 2^40 of them neither overflow nor vanish.  The sum's order (another one
// where `norms` is given) shows in the 32-bit result only where that lies a
// 64-bit rounding from the middle between two numbers.  No atomics on sums: block b's part of tensor k
// goes to slot b + k (along the walk over (b, k) one of the two grows at each
// part, so no two parts share a slot), and the block that finishes last adds
// the slots in a fixed order, whichever block that is.
//
// Bound by HBM: 134M fp16 values in 44.8 us (6.0 TB/s of the 6.55 that a copy
// reaches), 16.8M fp32 in 13.8 (4.9); conversions and sums in 64 bits hide
// behind the loads (probed: 77 us for 134M fp32 in either width).  What stays
// is 3.9 us for the smallest list: launch, first loads, the last block's round
// trips (its ticket, the slots).  A second launch for the finish took 6.2.
// ---------------------------------------------------------------------------
enum { kL1 = SPIN4D_NORM_L1, kL2 = SPIN4D_NORM_L2, kMax = SPIN4D_NORM_MAX };
constexpr int kWarps = kThreads / 32;
constexpr int kParts = 16;                    // tensors whose parts a block holds before it writes them out

template <int NORM>
__device__ __forceinline__ double join(double a, double b) {
  if (NORM == kMax) return (a > b || isnan(a)) ? a : b;   // a NaN stays
  return a + b;
}
template <int NORM>
__device__ __forceinline__ void take(const float x[kVec], double acc[2]) {
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
    const double d = (double)x[j];
    acc[j & 1] = NORM == kL2 ? fma(d, d, acc[j & 1]) : join<NORM>(acc[j & 1], fabs(d));
  }
}
template <int NORM, int LANES>
__device__ __forceinline__ double lanes_join(double a) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) a = join<NORM>(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// This thread's part of tiles [t, stop) of one tensor.
template <int NORM, int BYTES>
__device__ __forceinline__ double norm_of_tiles(const void* a, const Meta meta, uint32_t t, uint32_t stop) {
  constexpr int kAhead = 16 / BYTES;          // 32 registers of loads in flight
  double acc[2] = {0.0, 0.0};
  const int64_t n = meta.n();
  const int shift = meta.shift();
  const bool bf = meta.dtype() == SPIN4D_BF16;
  const uint32_t head = t == 0 && shift != 0;                            // the first tile begins below index 0
  const uint32_t whole = (uint32_t)min((uint64_t)stop, (uint64_t)(n + shift) / kTile);   // from here on it is partial
  t += head;
  const char* at = static_cast<const char*>(a) + ((int64_t)t * kTile + threadIdx.x * kVec - shift) * BYTES;
  for (; t + kAhead <= whole; t += kAhead, at += kAhead * kTile * BYTES) {
    Raw<BYTES> r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const char* const from = at + u * kTile * BYTES;
      const Places q(t + u, shift, n);
      if (expect(q.whole && from == static_cast<const char*>(a) + q.first * BYTES && q.vector_in(a, BYTES)))
        load_raw<kKeep>(from, r[u]);
      else
        fetch<kKeep>(a, q, r[u], true);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float x[kVec];
      unpack(r[u], bf, x);
      take<NORM>(x, acc);
    }
  }
  // the first tile, those left over, the last
  const uint32_t rest = head + (stop - t);
  for (uint32_t i = 0; i < rest; i += 4) {
    Raw<BYTES> r[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (i + u < rest) {
        fetch<kKeep>(a, Places(i + u < head ? 0u : t + (i + u - head), shift, n), r[u]);
      } else {
#pragma unroll
        for (int j = 0; j < kVec * BYTES / 4; ++j) r[u].w[j] = 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float x[kVec];
      unpack(r[u], bf, x);
      take<NORM>(x, acc);
    }
  }
  return join<NORM>(acc[0], acc[1]);
}

struct NormArgs {
  double grad_scale, max_norm;
  int first, last;                            // launch of the list
  spin4d_grad_control* control;
  float* norms;                               // this launch's tensors' (may be null)
  double* total;                              // carried from launch to launch of one list
  double* slots;
};

// A kernel parameter read lane by lane: through its address, as memory, where the constant bank would
// serve one lane at a time.
template <typename T>
__device__ __forceinline__ const T* as_memory(const T* p) {
  asm volatile("" : "+l"(p));
  return p;
}

template <int CAP, int NORM>
__global__ void __launch_bounds__(kThreads, kNormBlocks) norm_kernel(const __grid_constant__ List<NormEntry, CAP> list,
                                                                     const NormArgs f) {
  __shared__ double part[kParts][kWarps];
  __shared__ int part_slot[kParts];
  __shared__ bool is_last;
  __shared__ double sums[kMaxNormBlocks + CAP];
  __shared__ uint32_t tile0[CAP > 16 ? CAP + 1 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t per = list.per;
  uint32_t t = blockIdx.x * per;
  const uint32_t end = min(list.tiles, t + per);
  const int owner = list.owner(t);
  if (t < end) {
    const NormEntry& e = list.at[owner];
    for (uint32_t i = t; i < min(end, t + 4); ++i)
      warm(e.a, Places(i - list.tile0[owner], e.meta.shift(), e.meta.n()), dtype_bytes(e.meta.dtype()));
  }
  pdl_wait();
  pdl_release();
  const int slots = list.tiles == 0 ? 0 : gridDim.x + (f.norms ? list.count - 1 : 0);
  double acc = 0.0;
  int parts = 0;
  // the warps walk through the block's tensors on their own; they meet when the parts are written out
  auto write_parts = [&]() {
    __syncthreads();
    if (threadIdx.x < parts) {
      double s = part[threadIdx.x][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s = join<NORM>(s, part[threadIdx.x][w]);
      // (a list without values has one block, whose slot nobody reads)
      if (expect(part_slot[threadIdx.x] >= 0 && part_slot[threadIdx.x] < max(slots, 1))) f.slots[part_slot[threadIdx.x]] = s;
    }
    __syncthreads();
    parts = 0;
  };
  for (int k = owner; t < end && expect(k < list.count); ++k) {
    const uint32_t base = list.tile0[k], stop = min(end, list.tile0[k + 1]);
    if (t >= stop) continue;                  // a tensor without values
    const void* a = list.at[k].a;
    const Meta meta = list.at[k].meta;
    // its last tiles may be there only for balance
    const uint32_t real = (uint32_t)((meta.n() + meta.shift() + kTile - 1) / kTile);
    double one = 0.0;
    if (t - base < real) {
      if (meta.dtype() == SPIN4D_F32) one = norm_of_tiles<NORM, 4>(a, meta, t - base, min(stop - base, real));
      else one = norm_of_tiles<NORM, 2>(a, meta, t - base, min(stop - base, real));
    }
    t = stop;
    if (f.norms) {
      one = lanes_join<NORM, 32>(one);
      if (lane == 0) part[parts][warp] = one;
      if (threadIdx.x == 0) part_slot[parts] = blockIdx.x + k;
      if (++parts == kParts) write_parts();
    } else {
      acc = join<NORM>(acc, one);
    }
  }
  if (!f.norms) {                             // only the whole is asked for: one slot for each block
    acc = lanes_join<NORM, 32>(acc);
    if (lane == 0) part[0][warp] = acc;
    if (threadIdx.x == 0) part_slot[0] = blockIdx.x;
    parts = 1;
  }
  write_parts();
  // The last block to arrive finishes.  The ticket wraps to 0 for the next launch.
  if (threadIdx.x == 0) {
    uint32_t was;
    asm volatile("atom.acq_rel.gpu.global.inc.u32 %0, [%1], %2;"
                 : "=r"(was)
                 : "l"(&f.control->ticket), "r"(gridDim.x - 1)
                 : "memory");
    is_last = was == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  // All slots at once into shared memory: what follows is sums of few terms in a fixed order.
  constexpr int kSlotLoads = (kMaxNormBlocks + CAP + kThreads - 1) / kThreads;
  constexpr int kTileLoads = CAP > 16 ? CAP / kThreads + 1 : 0;
  const int starts = f.norms ? list.count + 1 : 0;
  double slot[kSlotLoads];
  uint32_t start[kTileLoads + 1];
#pragma unroll
  for (int j = 0; j < kSlotLoads; ++j) {
    const int i = threadIdx.x + j * kThreads;
    slot[j] = i < slots ? __ldcg(&f.slots[i]) : 0.0;
  }
  const uint32_t* from = as_memory(list.tile0);
#pragma unroll
  for (int j = 0; j < kTileLoads; ++j) {
    const int k = threadIdx.x + j * kThreads;
    start[j] = k < starts ? from[k] : 0u;
  }
  int32_t step = 0, skipped = 0;
  if (threadIdx.x == 0) {
    step = f.control->step;
    skipped = f.control->skipped;
  }
#pragma unroll
  for (int j = 0; j < kSlotLoads; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < slots) sums[i] = slot[j];
  }
#pragma unroll
  for (int j = 0; j < kTileLoads; ++j) {
    const int k = threadIdx.x + j * kThreads;
    if (k < starts) tile0[k] = start[j];
  }
  __syncthreads();
  double mine = 0.0;
  auto finish_tensor = [&](int k, double s) {
    f.norms[k] = (float)(f.grad_scale * (NORM == kL2 ? sqrt(s) : s));
    mine = join<NORM>(mine, s);
  };
  auto slot_sum = [&](int i) { return expect(i >= 0 && i < slots) ? sums[i] : 0.0; };
  auto by_warp = [&](int k, uint32_t a, uint32_t e) {
    double s = 0.0;
    if (e > a) {
      const int b1 = (e - 1) / per;
      for (int b = a / per + lane; b <= b1; b += 32) s = join<NORM>(s, slot_sum(b + k));
    }
    s = lanes_join<NORM, 32>(s);
    if (lane == 0) finish_tensor(k, s);
  };
  if (!f.norms) {
    for (int i = threadIdx.x; i < slots; i += kThreads) mine = join<NORM>(mine, sums[i]);
  } else if (CAP <= 16) {
    for (int k = warp; k < list.count; k += kWarps) by_warp(k, list.tile0[k], list.tile0[k + 1]);
  } else {
    // a thread for each tensor of few slots, a warp for each of the (few) others
    for (int k = threadIdx.x; k < list.count; k += kThreads) {
      const uint32_t a = tile0[k], e = tile0[k + 1];
      if (e - a > 8 * per) continue;
      double s = 0.0;
      if (e > a) {
        const int b1 = (e - 1) / per;
        for (int b = a / per; b <= b1; ++b) s = join<NORM>(s, slot_sum(b + k));
      }
      finish_tensor(k, s);
    }
    for (int k0 = warp * 32; k0 < list.count; k0 += kThreads) {
      const bool is_long = k0 + lane < list.count && tile0[k0 + lane + 1] - tile0[k0 + lane] > 8 * per;
      for (uint32_t todo = __ballot_sync(0xffffffffu, is_long); todo; todo &= todo - 1) {
        const int k = k0 + __ffs(todo) - 1;
        by_warp(k, tile0[k], tile0[k + 1]);
      }
    }
  }
  mine = lanes_join<NORM, 32>(mine);
  if (lane == 0) part[0][warp] = mine;
  __syncthreads();
  if (warp != 0) return;
  double total = lanes_join<NORM, kWarps>(part[0][lane % kWarps]);
  if (lane != 0) return;
  if (!f.first) total = join<NORM>(*f.total, total);
  if (!f.last) {
    *f.total = total;
    return;
  }
  const double norm = f.grad_scale * (NORM == kL2 ? sqrt(total) : total);
  const float norm32 = (float)norm;
  const bool fine = isfinite(norm32);
  f.control->norm = norm32;
  f.control->coef = fine ? (float)(f.grad_scale * fmin(1.0, f.max_norm / (norm + 1e-6))) : 0.0f;
  if (fine) f.control->step = step + 1;
  else f.control->skipped = skipped + 1;
}

// ---------------------------------------------------------------------------
// Clip: out = coef * gradient.  Bound by HBM, or by L2 where the norm has just
// brought the gradient there: norm and clip of 11.5M fp32 values (46 MB in, 46
// out) 23.5 us, of 33M 67.4, which at 3 x 4 bytes a value is 5.9 TB/s.
// ---------------------------------------------------------------------------
// Tiles [t, stop) of one tensor, from the last down.
template <int BYTES>
__device__ __forceinline__ void clip_tiles(const void* a, void* o, const Meta meta, uint32_t t, uint32_t stop, float coef) {
  constexpr int kAhead = 4 / BYTES;           // 8 registers of loads in flight; the blocks are many
  const int64_t n = meta.n();
  const int shift = meta.shift();
  while (stop > t) {
    Raw<BYTES> r[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (stop - t > u) fetch<kStream>(a, Places(stop - 1 - u, shift, n), r[u], meta.loose());
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (stop - t > u) {
        float x[kVec];
        unpack(r[u], meta.dtype() == SPIN4D_BF16, x);
#pragma unroll
        for (int i = 0; i < kVec; ++i) x[i] = coef == 0.0f ? 0.0f : coef * x[i];   // zeros whatever the gradient holds
        // kept: the optimiser reads it next (norm, clip and Adam of 4M values 28.9 us, streamed 30.0)
        put(o, meta.out_dtype(), Places(stop - 1 - u, shift, n), x);
      }
    stop -= min((uint32_t)kAhead, stop - t);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) clip_kernel(const __grid_constant__ List<ClipEntry, CAP> list,
                                                           const spin4d_grad_control* control) {
  pdl_wait();
  pdl_release();
  const uint32_t begin = (gridDim.x - 1 - blockIdx.x) * list.per;
  uint32_t end = min(list.tiles, begin + list.per);
  const float coef = control->coef;
  for (int k = list.owner(end - 1); end > begin && expect(k >= 0); --k) {
    const uint32_t base = list.tile0[k], t = max(begin, base);
    if (t >= end) continue;                   // a tensor without values
    const ClipEntry& e = list.at[k];
    // in place and within bounds, as in most steps: every value would be written back as it is (norm and clip of 16.8M
    // fp32 values 19.3 us, with a coefficient below 1 31.4)
    if (coef != 1.0f || e.out != e.a) {
      if (e.meta.dtype() == SPIN4D_F32) clip_tiles<4>(e.a, e.out, e.meta, t - base, end - base, coef);
      else clip_tiles<2>(e.a, e.out, e.meta, t - base, end - base, coef);
    }
    end = t;
  }
}

// ---------------------------------------------------------------------------
// Adam with decoupled weight decay, formula in the header.  Four streams in,
// three and the working copy out: bound by HBM, 134M parameters with fp16
// copies (30 bytes each) in 595 us, 6.8 TB/s; 16.8M in 74.  72 to 74 registers for 128
// bytes of loads a thread, three blocks a SM; the first loads are on their way
// before the control block is read, and in L2 before the norm has ended.
// ---------------------------------------------------------------------------
// The square root within 2^-23 of itself (subnormal arguments too).  With it and a quotient within 2 ulp a step
// is off by at most 2^-22 of what it moves a parameter more than with the correctly rounded ones, of which the
// parameter's own rounding usually leaves nothing.  Those took most of the kernel's instructions, and more where
// the state of untouched entries has decayed below 2^-126.  Norm and update with them of the smallest decoder 7.8 us, of
// 200 tensors 15.8, of 16.8M parameters 89 to 105, of 134M 693 to 746; so 6.0, 13.2, 87 and 687 (from graphs).
__device__ __forceinline__ float root(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct AdamArgs {
  float b1, b2, omb1, omb2, eps;
  double log_b1, log_b2;                      // for a step that only the device knows
  int step;                                   // 0: the control's
  int zero_grad;
  const spin4d_grad_control* control;         // may be null
  int32_t* flag;                              // may be null
};

template <int CAP>
__global__ void __launch_bounds__(kThreads, 3) adam_list_kernel(const __grid_constant__ List<AdamEntry, CAP> list,
                                                                const AdamArgs a) {
  const uint32_t begin = (gridDim.x - 1 - blockIdx.x) * list.per;
  uint32_t end = min(list.tiles, begin + list.per);
  const int last = list.owner(end - 1);
  {
    const AdamEntry& e = list.at[last];
    const Places q(end - 1 - list.tile0[last], e.meta.shift(), e.meta.n());
    warm(e.p, q, 4);
    warm(e.m, q, 4);
    warm(e.v, q, 4);
  }
  pdl_wait();
  pdl_release();
  float coef = 1.0f, inv_bc1 = 0.0f, inv_bc2 = 0.0f;
  bool ready = false, skip = false, bad = false;
  for (int k = last; end > begin && expect(k >= 0); --k) {
    const uint32_t base = list.tile0[k], stop = max(begin, base);
    if (stop >= end) continue;                // a tensor without values
    const AdamEntry& e = list.at[k];
    for (uint32_t t = end; t-- > stop;) {
      const Places q(t - base, e.meta.shift(), e.meta.n());
      Raw<4> rp, rm, rv, rg;
      fetch<kKeep>(e.p, q, rp);
      fetch<kKeep>(e.m, q, rm);
      fetch<kKeep>(e.v, q, rv);
      if (e.meta.dtype() == SPIN4D_F32) fetch<kKeep>(e.g, q, rg, e.meta.loose());
      else fetch<kKeep>(e.g, q, reinterpret_cast<Raw<2>&>(rg), e.meta.loose());
      if (!ready) {                           // behind the first loads, which do not wait for it
        ready = true;
        int step = a.step;
        if (a.control) {
          coef = a.control->coef;
          if (step == 0) step = a.control->step;
          skip = !isfinite(a.control->norm) || step < 1;
        }
        // 1 - b^step = -expm1(step log b): the product in 64 bits, then within 2 ulp of fp32
        inv_bc1 = 1.0f / -expm1f((float)(step * a.log_b1));
        inv_bc2 = 1.0f / -expm1f((float)(step * a.log_b2));
      }
      if (skip && !a.zero_grad) return;       // (the flag stays as it is)
      if (!skip) {
        float g[kVec], p[kVec], m[kVec], v[kVec];
        unpack(rp, false, p);
        unpack(rm, false, m);
        unpack(rv, false, v);
        if (e.meta.dtype() == SPIN4D_F32) unpack(rg, false, g);
        else unpack(reinterpret_cast<Raw<2>&>(rg), e.meta.dtype() == SPIN4D_BF16, g);
        const float lr = e.lr, decay = lr * e.decay;
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float gi = coef == 0.0f ? 0.0f : coef * g[i];
          m[i] = a.b1 * m[i] + a.omb1 * gi;
          v[i] = a.b2 * v[i] + a.omb2 * (gi * gi);
          const float mh = m[i] * inv_bc1, vh = v[i] * inv_bc2;
          // outside [0, n) all four are 0: with eps = 0 the quotient is NaN there, which neither is stored nor flagged
          p[i] -= __fdividef(lr * mh, root(vh) + a.eps) + decay * p[i];
        }
        if (a.flag) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) bad |= !isfinite(p[i]) && (q.whole || q.has(i));
        }
        put(e.p, SPIN4D_F32, q, p);
        put(e.m, SPIN4D_F32, q, m);
        put(e.v, SPIN4D_F32, q, v);
        if (e.work) {
          Raw<2> w;
          pack(p, e.meta.out_dtype() == SPIN4D_BF16, w);
          put(e.work, q, w);
        }
      }
      if (a.zero_grad) {
        const float zero[kVec] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        put(e.g, e.meta.dtype(), q, zero);
      }
    }
    end = stop;
  }
  if (a.flag && __syncthreads_or(bad) && threadIdx.x == 0) atomicExch(a.flag, 1);
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
bool dtype_ok(int dt) { return dt == SPIN4D_F32 || dt == SPIN4D_F16 || dt == SPIN4D_BF16; }

bool array_ok(const void* p, int64_t n, int bytes) { return n == 0 || (p && ((uintptr_t)p & (bytes - 1)) == 0); }

// A stretch of memory that a call reads or writes.
struct Stretch {
  uintptr_t lo = 0, hi = 0;
  bool write = false;
  Stretch() = default;
  Stretch(const void* p, int64_t n, int bytes, bool write_)
      : lo(p ? (uintptr_t)p : 0), hi(p ? (uintptr_t)p + (uint64_t)n * bytes : 0), write(write_) {}
  bool empty() const { return lo == hi; }
};

// Whether something that a call writes is also another array's: blocks run in no order, so the result would have
// none.  get(k, f) is the stretch of tensor k in family f (its parameters, its gradient, ...).  Families are
// nearly always in the order of their addresses and apart from one another, which one look over them shows;
// else all stretches are sorted.  True also when the host has no memory for that.
template <int FAMILIES, typename Get>
bool clash(int count, Get get) {
  const auto before = [](const Stretch& a, const Stretch& b) { return a.lo < b.lo; };
  Stretch box[FAMILIES];                      // what a family spans so far
  bool apart = true;
  for (int k = 0; k < count && apart; ++k)
    for (int f = 0; f < FAMILIES; ++f) {
      const Stretch s = get(k, f);
      if (s.empty()) continue;
      if (box[f].hi == 0) box[f].lo = s.lo;
      apart = apart && s.lo >= box[f].hi;
      box[f].hi = s.hi;
    }
  if (apart) {
    std::sort(box, box + FAMILIES, before);
    uintptr_t any = 0;
    for (const Stretch& s : box) {
      if (s.empty()) continue;
      apart = apart && s.lo >= any;
      any = s.hi;
    }
    if (apart) return false;
  }
  Stretch local[320];
  const size_t most = (size_t)FAMILIES * count;
  Stretch* const at = most <= 320 ? local : new (std::nothrow) Stretch[most];
  if (!at) return true;
  int used = 0;
  for (int k = 0; k < count; ++k)
    for (int f = 0; f < FAMILIES; ++f) {
      const Stretch s = get(k, f);
      if (!s.empty()) at[used++] = s;
    }
  std::sort(at, at + used, before);
  uintptr_t any = 0, written = 0;
  bool found = false;
  for (int i = 0; i < used && !found; ++i) {
    found = at[i].lo < (at[i].write ? any : written);
    any = std::max(any, at[i].hi);
    if (at[i].write) written = std::max(written, at[i].hi);
  }
  if (at != local) delete[] at;
  return found;
}

int shift_of(const void* p, int bytes) { return (int)(((uintptr_t)p & (kVec * bytes - 1)) >> (bytes == 4 ? 2 : 1)); }

// Appends a tensor's tiles; the callers have checked that a list's sum fits.
void add_tiles(uint32_t* tile0, int k, int64_t n, int shift) {
  tile0[k + 1] = tile0[k] + (n == 0 ? 0u : (uint32_t)((uint64_t)(n + (shift == kStrided ? 0 : shift) + kTile - 1) / kTile));
}

// Splits the list over at most `most` blocks; returns how many.
template <typename Entry, int CAP>
int split(List<Entry, CAP>& list, int most) {
  list.tiles = list.tile0[list.count];
  list.per = std::max(1u, (list.tiles + most - 1) / most);
  list.hint_shift = 0;
  if (CAP > 16) {
    while ((list.tiles >> list.hint_shift) >= (uint32_t)kHints) ++list.hint_shift;
    int k = 0;
    for (int h = 0; h <= kHints; ++h) {
      const uint64_t tile = (uint64_t)h << list.hint_shift;
      while (k + 1 < list.count && list.tile0[k + 1] <= tile) ++k;
      list.hint[h] = (uint16_t)k;
    }
  }
  return (int)std::max(1u, (list.tiles + list.per - 1) / list.per);
}

// launch_pdl without copies of the list on the way.
template <typename Kernel, typename... Args>
int launch(Kernel kernel, int blocks, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  void* list[] = {const_cast<void*>(static_cast<const void*>(&args))...};
  return cuda_status(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), list));
}

template <int CAP, int NORM>
int norm_launches(const spin4d_grad_tensor* ts, int count, NormArgs f, cudaStream_t s) {
  float* norms = f.norms;
  int at = 0;
  do {
    List<NormEntry, CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_grad_tensor& t = ts[at + k];
      const int shift = shift_of(t.grad, dtype_bytes(t.grad_dtype));
      list.at[k] = {t.grad, meta_of(t.n, t.grad_dtype, 0, shift, false)};
      add_tiles(list.tile0, k, t.n, shift);
    }
    const int most = std::min(kNormBlocks * sm_count(), kMaxNormBlocks);
    // A block that begins another tensor waits for its first values once more, about kTensorTiles tiles' time:
    // where blocks have several tiles, a tensor of a long list counts for that many more.  (16.8M fp16 values
    // and 40 tensors of up to 20000: 12.5 us with 4, 11.6 with 6; 33M fp32 and 300 of them 25.1 and 24.7.  With
    // 4 blocks a SM and a longer finish it was 22.2 us without, 14.4 with 3.)
    if (CAP > 16 && list.tile0[list.count] > (uint32_t)most) {
      uint32_t more = 0;
      for (int k = 0; k < list.count; ++k) {
        const bool some = list.at[k].meta.n() > 0;
        if (some) more += kTensorTiles;
        list.tile0[k + 1] += more;
      }
    }
    const int blocks = split(list, most);
    f.first = at == 0;
    f.last = at + list.count == count;
    f.norms = norms ? norms + at : nullptr;
    SPIN4D_CHECK(launch(norm_kernel<CAP, NORM>, blocks, s, list, f));
    at += list.count;
  } while (at < count);
  return SPIN4D_OK;
}

// A launch costs the host by the size of its parameters, and the norm's finish by the capacity: lists have the smallest
// capacity that holds them.  The largest fill what a launch can carry (32 KB).  The steps below them, us a call through
// the binding (the next larger capacity in brackets): norm of 16 tensors 4.9, of 40 5.2 (5.2), of 65 5.4 (5.8), of 300
// 7.1 (7.65); clip of 2 3.1 (with the largest 4.3), of 40 3.7 (3.9), of 65 4.0 (4.7), of 300 5.4 (6.1); Adam of 40 5.4
// (5.6), of 65 5.9 (6.4), of 200 7.5 (7.8).  320 keeps clip's parameters below 10 KB, 224 is half of Adam's largest.
template <int NORM>
int norm_list(const spin4d_grad_tensor* ts, int count, const NormArgs& f, cudaStream_t s) {
  if (count <= 16) return norm_launches<16, NORM>(ts, count, f, s);
  if (count <= 64) return norm_launches<64, NORM>(ts, count, f, s);
  if (count <= 320) return norm_launches<320, NORM>(ts, count, f, s);
  return norm_launches<kNormCap, NORM>(ts, count, f, s);
}

template <int CAP>
int clip_launches(const spin4d_grad_tensor* ts, int count, const spin4d_grad_control* control, cudaStream_t s) {
  for (int at = 0; at < count; at += CAP) {
    List<ClipEntry, CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_grad_tensor& t = ts[at + k];
      void* out = t.out ? t.out : const_cast<void*>(t.grad);
      const int out_dtype = t.out ? t.out_dtype : t.grad_dtype;
      const int shift = shift_of(out, dtype_bytes(out_dtype));
      const bool loose = shift != shift_of(t.grad, dtype_bytes(t.grad_dtype));
      list.at[k] = {t.grad, out, meta_of(t.n, t.grad_dtype, out_dtype, shift, loose)};
      add_tiles(list.tile0, k, t.n, shift);
    }
    const int blocks = split(list, kClipBlocks * sm_count());
    if (!list.tiles) continue;
    SPIN4D_CHECK(launch(clip_kernel<CAP>, blocks, s, list, control));
  }
  return SPIN4D_OK;
}

template <int CAP>
int adam_launches(const spin4d_adam_tensor* ts, int count, const AdamArgs& a, cudaStream_t s) {
  for (int at = 0; at < count; at += CAP) {
    List<AdamEntry, CAP> list;
    list.count = std::min(CAP, count - at);
    list.tile0[0] = 0;
    for (int k = 0; k < list.count; ++k) {
      const spin4d_adam_tensor& t = ts[at + k];
      int shift = shift_of(t.params, 4);
      const bool loose = shift != shift_of(t.grad, dtype_bytes(t.grad_dtype));
      if (shift != shift_of(t.m, 4) || shift != shift_of(t.v, 4) ||
          (t.params_work && shift != shift_of(t.params_work, 2)) || (loose && a.zero_grad))
        shift = kStrided;
      list.at[k] = {t.params, t.m, t.v, t.grad, t.params_work,
                    meta_of(t.n, t.grad_dtype, t.work_dtype & 15, shift, loose), t.lr, t.weight_decay};
      add_tiles(list.tile0, k, t.n, shift);
    }
    const int blocks = split(list, kAdamBlocks * sm_count());
    if (!list.tiles) continue;
    SPIN4D_CHECK(launch(adam_list_kernel<CAP>, blocks, s, list, a));
  }
  return SPIN4D_OK;
}

}  // namespace
}  // namespace spin4d

using namespace spin4d;

extern "C" size_t spin4d_grad_norm_workspace(int count) {
  if (count < 0 || count > kMaxTensors) return 0;
  return sizeof(double) * (1 + kMaxNormBlocks + kNormCap);
}

extern "C" int spin4d_grad_norm(const spin4d_grad_tensor* tensors, int count, int norm_type, double grad_scale,
                                double max_norm, spin4d_grad_control* control, float* norms, void* workspace,
                                size_t ws_bytes, spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (norm_type != kL1 && norm_type != kL2 && norm_type != kMax) return SPIN4D_ERR_INVALID;
  // as the coefficient holds it: infinite it would make NaN of a zero gradient, 0 is the one that drops a gradient
  const float scale32 = (float)grad_scale;
  if (!(scale32 > 0.0f) || !isfinite(scale32) || !(max_norm >= 0.0)) return SPIN4D_ERR_INVALID;
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
  NormArgs f = {};
  f.grad_scale = grad_scale;
  f.max_norm = max_norm;
  f.control = control;
  f.norms = norms;
  f.total = static_cast<double*>(workspace);
  f.slots = static_cast<double*>(workspace) + 1;
  const cudaStream_t s = (cudaStream_t)stream;
  if (norm_type == kL2) return norm_list<kL2>(tensors, count, f, s);
  if (norm_type == kL1) return norm_list<kL1>(tensors, count, f, s);
  return norm_list<kMax>(tensors, count, f, s);
}

extern "C" int spin4d_clip_grads(const spin4d_grad_tensor* tensors, int count, const spin4d_grad_control* control,
                                 spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (!control || !aligned(control, 16)) return SPIN4D_ERR_INVALID;
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    const spin4d_grad_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxValues || !dtype_ok(t.grad_dtype) || (t.n && t.out && !dtype_ok(t.out_dtype)))
      return SPIN4D_ERR_INVALID;
    if (!array_ok(t.grad, t.n, dtype_bytes(t.grad_dtype))) return SPIN4D_ERR_INVALID;
    if (t.out && !array_ok(t.out, t.n, dtype_bytes(t.out_dtype))) return SPIN4D_ERR_INVALID;
    tiles += t.n / kTile + 2;
  }
  if (tiles >= (int64_t(1) << 31)) return SPIN4D_ERR_INVALID;
  const auto stretch = [tensors](int k, int f) {
    const spin4d_grad_tensor& t = tensors[k];
    const bool in_place = !t.out || (t.out == t.grad && t.out_dtype == t.grad_dtype);
    if (f == 0) return Stretch(t.grad, t.n, dtype_bytes(t.grad_dtype), in_place);
    return in_place ? Stretch() : Stretch(t.out, t.n, dtype_bytes(t.out_dtype), true);
  };
  if (clash<2>(count, stretch)) return SPIN4D_ERR_INVALID;
  if (fault_injected("spin4d_clip_grads")) return SPIN4D_ERR_INJECTED;
  if (count <= 16) return clip_launches<16>(tensors, count, control, (cudaStream_t)stream);
  if (count <= 64) return clip_launches<64>(tensors, count, control, (cudaStream_t)stream);
  if (count <= 320) return clip_launches<320>(tensors, count, control, (cudaStream_t)stream);
  return clip_launches<1024>(tensors, count, control, (cudaStream_t)stream);
}

extern "C" int spin4d_adam_step_tensors(const spin4d_adam_tensor* tensors, int count, int step, double b1, double b2,
                                        double eps, int zero_grad, const spin4d_grad_control* control,
                                        int32_t* nonfinite_flag, spin4d_stream_t stream) {
  if (count < 0 || count > kMaxTensors || (count > 0 && !tensors)) return SPIN4D_ERR_INVALID;
  if (step < 0 || (step == 0 && !control)) return SPIN4D_ERR_INVALID;
  // as the kernel holds them: a rate that rounds to 1 would never forget
  if (!(b1 >= 0.0 && (float)b1 < 1.0f && b2 >= 0.0 && (float)b2 < 1.0f && eps >= 0.0)) return SPIN4D_ERR_INVALID;
  // the quotient holds to its bound for denominators from 2^-126 to 2^126, of which the root takes up to 2^64
  const float eps32 = (float)eps;
  if (eps32 != 0.0f && !(eps32 >= 0x1p-126f && eps32 <= 0x1p125f)) return SPIN4D_ERR_INVALID;
  if ((control && !aligned(control, 16)) || (nonfinite_flag && !aligned(nonfinite_flag, 4))) return SPIN4D_ERR_INVALID;
  int64_t tiles = 0;
  for (int k = 0; k < count; ++k) {
    const spin4d_adam_tensor& t = tensors[k];
    if (t.n < 0 || t.n > kMaxValues || !isfinite(t.lr) || !isfinite(t.weight_decay)) return SPIN4D_ERR_INVALID;
    if (!dtype_ok(t.grad_dtype)) return SPIN4D_ERR_INVALID;
    if (t.n && t.params_work &&
        ((t.work_dtype != SPIN4D_F16 && t.work_dtype != SPIN4D_BF16) || !array_ok(t.params_work, t.n, 2)))
      return SPIN4D_ERR_INVALID;
    if (!array_ok(t.params, t.n, 4) || !array_ok(t.m, t.n, 4) || !array_ok(t.v, t.n, 4) ||
        !array_ok(t.grad, t.n, dtype_bytes(t.grad_dtype)))
      return SPIN4D_ERR_INVALID;
    tiles += t.n / kTile + 2;
  }
  if (tiles >= (int64_t(1) << 31)) return SPIN4D_ERR_INVALID;
  const auto stretch = [tensors, zero_grad](int k, int f) {
    const spin4d_adam_tensor& t = tensors[k];
    switch (f) {
      case 0: return Stretch(t.params, t.n, 4, true);
      case 1: return Stretch(t.m, t.n, 4, true);
      case 2: return Stretch(t.v, t.n, 4, true);
      case 3: return Stretch(t.params_work, t.n, 2, true);
      default: return Stretch(t.grad, t.n, dtype_bytes(t.grad_dtype), zero_grad != 0);
    }
  };
  if (clash<5>(count, stretch)) return SPIN4D_ERR_INVALID;
  if (fault_injected("spin4d_adam_step_tensors")) return SPIN4D_ERR_INJECTED;
  AdamArgs a;
  a.b1 = (float)b1;
  a.b2 = (float)b2;
  a.omb1 = (float)(1.0 - b1);
  a.omb2 = (float)(1.0 - b2);
  a.eps = eps32;
  a.log_b1 = log(b1);
  a.log_b2 = log(b2);
  a.step = step;
  a.zero_grad = zero_grad ? 1 : 0;
  a.control = control;
  a.flag = nonfinite_flag;
  if (count <= 16) return adam_launches<16>(tensors, count, a, (cudaStream_t)stream);
  if (count <= 64) return adam_launches<64>(tensors, count, a, (cudaStream_t)stream);
  if (count <= 224) return adam_launches<224>(tensors, count, a, (cudaStream_t)stream);
  return adam_launches<448>(tensors, count, a, (cudaStream_t)stream);
}
