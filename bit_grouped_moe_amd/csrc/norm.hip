// Root-mean-square norm of rows, with the residual's addition before it and
// its result in 8 bits behind it, and its gradient.
//
//   forward   h = x + r, rounded to the rows' type;  n_i = h_i / sqrt(mean h^2 + eps)
//             y_i = n_i w_i, rounded once;  MXFP8 codes and scales of the unrounded y
//   backward  with g = dy w and rstd = 1 / sqrt(mean h^2 + eps):
//             dx_i = rstd (g_i - n_i mean(g n)) + dh_i,   dw_i = sum over rows dy_i n_i
//             (dh the gradient that reaches h by another way: dx is x's and r's)
//
// The norm is the norm of the rounded h, the value that is stored: a backward
// pass that reads h again differentiates what was computed.  Sums are float32:
// a lane's own elements in order, then DPP and LDS sums in a fixed order.
//
// Bound by HBM.  A row stays in registers between its sum and its results: each
// value is read once.  kWaves waves share a row, eight values a lane and step,
// kC steps; a quad of lanes so holds a block of 32 and quantises as the
// quantiser does.
#include <type_traits>

#include "gq_host.hpp"
#include "values.hpp"

namespace gq {

constexpr int kNormMaxWidth = 32768;

template <int kType>
constexpr int kTypeSize = kType == GQ_F32 ? 4 : 2;

template <int kType>
__device__ __forceinline__ float load_one(const void* p) {
  if constexpr (kType == GQ_F32) return *static_cast<const float*>(p);
  else if constexpr (kType == GQ_BF16)
    return __uint_as_float((uint32_t)*static_cast<const uint16_t*>(p) << 16);
  else return (float)*static_cast<const _Float16*>(p);
}
template <int kType>
__device__ __forceinline__ void store_one(void* p, float v) {
  if constexpr (kType == GQ_F32) *static_cast<float*>(p) = v;
  else if constexpr (kType == GQ_BF16) *static_cast<uint16_t*>(p) = f32_to_bf16_bits(v);
  else *static_cast<_Float16*>(p) = (_Float16)v;
}
template <int kType>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (kType == GQ_F32) return v;
  else if constexpr (kType == GQ_BF16) return (float)(__bf16)v;
  else return (float)(_Float16)v;
}
template <int kType>
__device__ __forceinline__ void store8(void* p, const float (&v)[8]) {
  if constexpr (kType == GQ_F32) {
    u32x4_a4* q = static_cast<u32x4_a4*>(p);
    q[0] = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                 __float_as_uint(v[3])};
    q[1] = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                 __float_as_uint(v[7])};
  } else if constexpr (kType == GQ_BF16) {
    *static_cast<u32x4_a2*>(p) = u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                       pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  } else {
    f16x8 h;
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
    *static_cast<u32x4_a2*>(p) = __builtin_bit_cast(u32x4, h);
  }
}

// Values [8 c, 8 c + 8) of a row of H: zeros past its end.  `row` is its address.
template <int kType>
__device__ __forceinline__ void load_chunk(const char* row, int c, int H, float (&v)[8]) {
  const char* p = row + (int64_t)c * 8 * kTypeSize<kType>;
  if (8 * c + 8 <= H) {
    load8<kType>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = 8 * c + i < H ? load_one<kType>(p + i * kTypeSize<kType>) : 0.f;
  }
}
// The same as stored, to be widened where it is used.
template <int kType>
struct Chunk {
  u32x4 a[kType == GQ_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* row, int c, int H) {
    const char* p = row + (int64_t)c * 8 * kTypeSize<kType>;
    if (8 * c + 8 <= H) {
      if constexpr (kType == GQ_F32) {
        a[0] = reinterpret_cast<const u32x4_a4*>(p)[0];
        a[1] = reinterpret_cast<const u32x4_a4*>(p)[1];
      } else {
        a[0] = *reinterpret_cast<const u32x4_a2*>(p);
      }
    } else {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (kType == GQ_F32)
          w[i] = 8 * c + i < H ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
        else
          w[i] = 8 * c + i < H ? (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] : 0u;
      }
      if constexpr (kType == GQ_F32) {
        a[0] = u32x4{w[0], w[1], w[2], w[3]};
        a[1] = u32x4{w[4], w[5], w[6], w[7]};
      } else {
        a[0] = u32x4{w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
      }
    }
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
    if constexpr (kType == GQ_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(a[i / 4][i % 4]);
    } else {
      widen8<kType>(a[0], v);
    }
  }
};
template <int kType>
__device__ __forceinline__ void store_chunk(char* row, int c, int H, const float (&v)[8]) {
  char* p = row + (int64_t)c * 8 * kTypeSize<kType>;
  if (8 * c + 8 <= H) {
    store8<kType>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * c + i < H) store_one<kType>(p + i * kTypeSize<kType>, v[i]);
  }
}

// Sums over the kWaves waves of a row, the same in every lane.  `turn` takes
// one half of `part` and then the other, so that one barrier a call is enough.
template <int kWaves, int kSums>
__device__ __forceinline__ void row_sums(float (&s)[kSums], float (*part)[kSums * 16], int turn) {
#pragma unroll
  for (int k = 0; k < kSums; ++k)
    s[k] = __int_as_float(
        __builtin_amdgcn_readlane(__float_as_int(group_sum_last(s[k], kWave)), kWave - 1));
  if constexpr (kWaves > 1) {
    const int wave = threadIdx.x / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) {
#pragma unroll
      for (int k = 0; k < kSums; ++k) part[turn][16 * k + wave] = s[k];
    }
    lds_barrier();
#pragma unroll
    for (int k = 0; k < kSums; ++k) {
      float t = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) t += part[turn][16 * k + w];
      s[k] = t;
    }
  }
}

struct NormArgs {
  const char* x;
  const char* residual;          // or null
  const char* weight;
  char* sum;                     // or null
  char* y;                       // or null
  u32x2* codes;                  // or null
  uint8_t* scales;
  u32x4* values;                 // or null
  int64_t rows, x_stride, r_stride;   // strides in bytes
  int H;
  float eps;
};

// Threads of a workgroup: as many rows as it has groups of kWaves waves.
template <int kWaves>
constexpr int kNormThreads = kWaves == 1 ? 256 : kWaves * kWave;

template <int kType, int kWType, int kWaves, int kC>
__global__ __launch_bounds__(kNormThreads<kWaves>) void rms_norm_kernel(NormArgs g) {
  constexpr int kLanes = kWaves * kWave;
  constexpr int kRows = kNormThreads<kWaves> / kLanes;
  __shared__ float part[2][16];
  const int lane = threadIdx.x & (kLanes - 1);
  const int H = g.H, chunks = (H + 7) / 8;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes; row < g.rows;
       row += (int64_t)gridDim.x * kRows) {
    float v[kC][8];
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = lane + j * kLanes;
      if (c < chunks) {
        load_chunk<kType>(g.x + row * g.x_stride, c, H, v[j]);
        if (g.residual) {
          float r[8];
          load_chunk<kType>(g.residual + row * g.r_stride, c, H, r);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = rounded<kType>(v[j][i] + r[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = __builtin_fmaf(v[j][i], v[j][i], s[0]);
      }
    }
    row_sums<kWaves, 1>(s, part, turn);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(s[0] / (float)H + g.eps);
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = lane + j * kLanes;
      if (c >= chunks) continue;
      if (g.sum) store_chunk<kType>(g.sum + row * H * kTypeSize<kType>, c, H, v[j]);
      float w[8], y[8];
      load_chunk<kWType>(g.weight, c, H, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[j][i] * rstd * w[i];
      if (g.y) store_chunk<kType>(g.y + row * H * kTypeSize<kType>, c, H, y);
      if (g.codes) {                                     // H % 32 == 0: whole quads
        uint32_t scale;
        const u32x2 q = quantize8_e4m3(y, scale);
        const int64_t o = row * chunks + c;
        g.codes[o] = q;
        if ((threadIdx.x & 3) == 0) g.scales[o >> 2] = (uint8_t)scale;
        if (g.values) g.values[o] = e4m3_bf16_scaled(q, scale);
      }
    }
  }
}

struct NormBackArgs {
  const char* dy;
  const char* h;
  const char* dh;                // or null
  const char* weight;
  char* dx;
  float* partial;                // [workgroups, H] or null: no gain gradient
  int64_t rows, dy_stride, h_stride, dh_stride;
  int H;
  float eps;
};

// A workgroup takes every gridDim.x-th group of rows and adds what its lanes'
// columns give to dw in registers; its sums go to one row of `partial`.  A row's
// loads go out before the row before it is worked on: a row is one memory latency
// and a barrier otherwise (16384 rows of 2048 in bf16, 73 us, so 48).
template <int kType, int kWType, int kWaves, int kC>
__global__ __launch_bounds__(kNormThreads<kWaves>) void rms_norm_backward_kernel(NormBackArgs g) {
  constexpr int kLanes = kWaves * kWave;
  constexpr int kRows = kNormThreads<kWaves> / kLanes;
  __shared__ float part[2][32];
  __shared__ float meet[kRows > 1 ? kRows - 1 : 1][kRows > 1 ? kLanes * 8 : 1];
  const int lane = threadIdx.x & (kLanes - 1);
  const int H = g.H, chunks = (H + 7) / 8;
  // what the registers hold: rows of one to four waves the next row's values too, of
  // sixteen waves and 32 values a lane not even this row's (they are read again).  The
  // 128 registers of 1024 threads do not quite do: bf16 rows of 8193 to 16384 values
  // spill 36 bytes a lane, float32 rows beyond 12
  constexpr bool kNext = kWaves < 16 && (kType != GQ_F32 || kC < 4), kKeep = kWaves * kC < 64;
  float acc[kC][8];
#pragma unroll
  for (int j = 0; j < kC; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.f;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kLanes;
  Chunk<kType> h[kC], dy[kC], dh[kC];
  Chunk<kWType> w[kC];
  auto fetch_one = [&](int64_t r, int j) {
    const int c = lane + j * kLanes;
    if (c < chunks) {
      h[j].load(g.h + r * g.h_stride, c, H);
      dy[j].load(g.dy + r * g.dy_stride, c, H);
      if (g.dh) dh[j].load(g.dh + r * g.dh_stride, c, H);
    }
  };
  auto fetch = [&](int64_t r) {
    r = r < g.rows ? r : g.rows - 1;
#pragma unroll
    for (int j = 0; j < kC; ++j) fetch_one(r, j);
  };
  auto gain = [&](int j) {
    if (lane + j * kLanes < chunks) w[j].load(g.weight, lane + j * kLanes, H);
  };
  if constexpr (kNext) fetch(row);
  if constexpr (kKeep) {
#pragma unroll
    for (int j = 0; j < kC; ++j) gain(j);
  }
  int turn = 0;
  for (; row < g.rows; row += step) {
    Chunk<kType> h0[kC], dy0[kC], dh0[kC];
    if constexpr (kKeep) {
      if constexpr (!kNext) fetch(row);
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        h0[j] = h[j];
        dy0[j] = dy[j];
        dh0[j] = dh[j];
      }
      if constexpr (kNext) fetch(row + step);
    }
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      if constexpr (!kKeep) {
        fetch_one(row, j);
        gain(j);
        h0[j] = h[j];
        dy0[j] = dy[j];
      }
      if (lane + j * kLanes < chunks) {
        float v[8], d[8], wf[8];
        h0[j].widen(v);
        dy0[j].widen(d);
        w[j].widen(wf);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          s[0] = __builtin_fmaf(v[i], v[i], s[0]);
          s[1] = __builtin_fmaf(v[i], d[i] * wf[i], s[1]);
        }
      }
    }
    row_sums<kWaves, 2>(s, part, turn);
    turn ^= 1;
    const float rstd = 1.0f / sqrtf(s[0] / (float)H + g.eps);
    const float mean = s[1] * rstd / (float)H;             // mean(g n)
#pragma unroll
    for (int j = 0; j < kC; ++j) {
      const int c = lane + j * kLanes;
      if constexpr (!kKeep) {
        asm volatile("" ::: "memory");                     // (the values are read again)
        fetch_one(row, j);
        gain(j);
        h0[j] = h[j];
        dy0[j] = dy[j];
        dh0[j] = dh[j];
      }
      if (c >= chunks) continue;
      float v[8], d[8], wf[8], o[8], t[8];
      h0[j].widen(v);
      dy0[j].widen(d);
      w[j].widen(wf);
      if (g.dh) dh0[j].widen(t);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = v[i] * rstd;
        o[i] = rstd * __builtin_fmaf(-n, mean, d[i] * wf[i]);
        if (g.dh) o[i] += t[i];
        acc[j][i] = __builtin_fmaf(d[i], n, acc[j][i]);
      }
      store_chunk<kType>(g.dx + row * H * kTypeSize<kType>, c, H, o);
    }
  }
  if (!g.partial) return;
  float* out = g.partial + (int64_t)blockIdx.x * H;
#pragma unroll
  for (int j = 0; j < kC; ++j) {
    const int c = lane + j * kLanes;
    if constexpr (kRows > 1) {
      // the workgroup's waves in order
      const int wave = threadIdx.x / kLanes;
      lds_barrier();
      if (wave > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) meet[wave - 1][kLanes * i + lane] = acc[j][i];
      }
      lds_barrier();
      if (wave > 0) continue;
#pragma unroll
      for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] += meet[k][kLanes * i + lane];
    }
    if (c < chunks) store_chunk<GQ_F32>(reinterpret_cast<char*>(out), c, H, acc[j]);
  }
}

// dw: the sums of the workgroups' rows, 16 columns a workgroup and 64 runs of rows
// side by side, then the runs in a fixed order.  (Bound by latency: columns 64 at a
// time and 16 runs took 12 us for 512 rows of 2048, this 6.)
constexpr int kGainCols = 16, kGainRuns = 64;
template <int kWType>
__global__ __launch_bounds__(kGainCols * kGainRuns) void rms_norm_gain_kernel(
    const float* __restrict__ partial, int groups, int H, char* __restrict__ dw) {
  __shared__ float meet[kGainRuns][kGainCols];
  const int col = threadIdx.x % kGainCols, run = threadIdx.x / kGainCols;
  const int i = blockIdx.x * kGainCols + col;
  float s = 0.f;
  if (i < H) {
#pragma unroll 8
    for (int r = run; r < groups; r += kGainRuns) s += partial[(int64_t)r * H + i];
  }
  meet[run][col] = s;
  lds_barrier();
  // (runs 4 k .. 4 k + 3 in the lanes of run k, then those sixteen in the first's)
  if (run < 16) s = (meet[4 * run][col] + meet[4 * run + 1][col]) +
                    (meet[4 * run + 2][col] + meet[4 * run + 3][col]);
  lds_barrier();
  if (run < 16) meet[run][col] = s;
  lds_barrier();
  if (run == 0 && i < H) {
#pragma unroll
    for (int k = 1; k < 16; ++k) s += meet[k][col];
    store_one<kWType>(dw + (int64_t)i * kTypeSize<kWType>, s);
  }
}

// f(waves a row, steps) for rows of H values.  A wave a row needs no barrier and many
// rows want few instructions a row; up to a row for each compute unit, a row's own
// latency counts and its values are spread over all the lanes there are.  bf16, us,
// forward and backward with the gain's gradient, fewer waves a row against more:
//   rows    1024 wide (1, 4 waves)    2880 (4, 16)            8192 (4, 16)
//      1    3.3 5.9   2.9 5.1         3.6  6.0   3.1  5.4     5.2  8.1   3.6  6.2
//    256    3.9 6.3   3.2 6.8         4.2  9.2   3.8  8.6     6.5 16.3   5.0 14.4
//    512    4.0 6.9   3.4 7.7         4.8 11.8   5.3 12.7     8.4 19.9   7.5 20.1
//   1024    4.3 8.0   4.5 8.7         6.1 13.4   8.2 13.9    12.5 23.2  14.3 24.7
// 16384 rows of 512: a wave a row 13.2 and 16.5, four 18.1 and 34.2; of 2048: one wave
// 43.3 and 47.8, four 41.1 and 47.7.
// float32 in the forms chosen, forward and backward with the gain's gradient: 16384
// rows of 512 22.1 and 24.1, of 2048 95 and 103, 2048 of 8192 45 and 53 (4 bytes of each
// of four tensors, 5.0 to 6.1 TB/s).  Few wide rows are held up by the partial sums, a
// row of them a workgroup: 1024 of 16384 50 and 69, 512 of 32768 48 and 106, without the
// gain's gradient 45 and 67.
constexpr int kNormFew = 256;
template <typename F>
static void by_row(int64_t rows, int H, F&& f) {
  auto go = [&](auto w, auto c) { f(w, c); };
  using std::integral_constant;
  const bool few = rows <= kNormFew;
  if (H <= 512) go(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (H <= 1024 && !few) go(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (H <= 2048) go(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (H <= 8192 && few) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (H <= 4096) go(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else if (H <= 8192) go(integral_constant<int, 4>{}, integral_constant<int, 4>{});
  else if (H <= 16384) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

// f(type of the rows, type of the gain); the gain's is the rows' or float32.
template <typename F>
static void by_types(int32_t dtype, int32_t wtype, F&& f) {
  using std::integral_constant;
  using F32 = integral_constant<int, GQ_F32>;
  using B16 = integral_constant<int, GQ_BF16>;
  using F16 = integral_constant<int, GQ_F16>;
  if (dtype == GQ_F32) f(F32{}, F32{});
  else if (dtype == GQ_BF16 && wtype == GQ_F32) f(B16{}, F32{});
  else if (dtype == GQ_BF16) f(B16{}, B16{});
  else if (wtype == GQ_F32) f(F16{}, F32{});
  else f(F16{}, F16{});
}

static int norm_checks(int32_t dtype, int32_t wtype, int64_t rows, int32_t H, float eps) {
  if (dtype != GQ_F32 && dtype != GQ_BF16 && dtype != GQ_F16) return kInvalid;
  if (wtype != dtype && wtype != GQ_F32) return kInvalid;
  if (rows < 0 || H < 1 || !(eps >= 0.f && eps < 3.4e38f)) return kInvalid;
  if (H > kNormMaxWidth) return kNotSupported;
  return kOk;
}
static bool strides_fit(int64_t rows, int64_t stride) {
  return rows == 0 || stride <= INT64_MAX / 8 / rows;
}
static int type_size(int32_t dtype) { return dtype == GQ_F32 ? 4 : 2; }
static bool element_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(type_size(dtype) - 1)) == 0;
}

// An output in place of an input that lies at another stride would overwrite rows
// that are still to be read.
static bool apart(const void* out, const void* in, int64_t rows, int64_t stride, int32_t H) {
  return !out || out != in || rows == 1 || stride == H;
}

// Workgroups of the backward pass: its partial sums are one row each.  (Two a compute
// unit: 16384 rows of 2048 in bf16 take 63 us with 256 workgroups, 47.7 with 512, 48.4
// with 1024; 2048 rows of 8192 30, 31.6 and 43.)
constexpr int64_t kBackGroups = 512;
static int64_t back_groups(int64_t rows, int H) {
  int64_t groups = 0;
  by_row(rows, H, [&](auto w, auto) {
    constexpr int kRows = kNormThreads<decltype(w)::value> / (decltype(w)::value * kWave);
    groups = ceil_div64(rows, kRows);
  });
  return groups < kBackGroups ? groups : kBackGroups;
}
// The most of them for up to that many rows.  (Rows of 513 to 1024 values are one to a
// workgroup up to kNormFew rows and four from there on: the number falls at that border
// and nowhere else.)
static int64_t most_back_groups(int64_t rows, int H) {
  const int64_t all = back_groups(rows, H);
  const int64_t few = back_groups(rows < kNormFew ? rows : kNormFew, H);
  return all > few ? all : few;
}

}  // namespace gq

extern "C" int gq_rms_norm(const void* x, int64_t x_stride, const void* residual,
                           int64_t residual_stride, int32_t dtype, int64_t rows, int32_t H,
                           const void* weight, int32_t weight_dtype, float eps, void* sum, void* y,
                           uint8_t* codes, uint8_t* scales, uint16_t* values,
                           hipStream_t stream) {
  using namespace gq;
  const int st = norm_checks(dtype, weight_dtype, rows, H, eps);
  if (st == kInvalid) return st;
  if (x_stride < H || (residual && residual_stride < H) || (sum && !residual)) return kInvalid;
  if ((codes && H % 32) || !codes != !scales || (values && !codes)) return kInvalid;
  if (st != kOk || rows == 0) return st;
  if (!x || !weight || !(sum || y || codes)) return kInvalid;
  if (!element_aligned(x, dtype) || !element_aligned(residual, dtype) ||
      !element_aligned(weight, weight_dtype) || !element_aligned(sum, dtype) ||
      !element_aligned(y, dtype) || !aligned16(codes) || !aligned16(values))
    return kInvalid;
  if (!strides_fit(rows, x_stride) || (residual && !strides_fit(rows, residual_stride)) ||
      !strides_fit(rows, H))
    return kNotSupported;
  if ((sum && sum == y) || !apart(sum, x, rows, x_stride, H) || !apart(y, x, rows, x_stride, H) ||
      !apart(sum, residual, rows, residual_stride, H) ||
      !apart(y, residual, rows, residual_stride, H))
    return kInvalid;
  const int size = type_size(dtype);
  NormArgs g{static_cast<const char*>(x), static_cast<const char*>(residual),
             static_cast<const char*>(weight), static_cast<char*>(sum), static_cast<char*>(y),
             reinterpret_cast<u32x2*>(codes), scales, reinterpret_cast<u32x4*>(values), rows,
             x_stride * size, residual_stride * size, H, eps};
  by_types(dtype, weight_dtype, [&](auto t, auto wt) {
    by_row(rows, H, [&](auto w, auto c) {
      constexpr int kWaves = decltype(w)::value, kThreads = kNormThreads<kWaves>;
      const int64_t groups = ceil_div64(rows, kThreads / (kWaves * kWave));
      const int64_t most = most_groups(kThreads);
      hipLaunchKernelGGL((rms_norm_kernel<decltype(t)::value, decltype(wt)::value, kWaves,
                                          decltype(c)::value>),
                         dim3((unsigned)(groups < most ? groups : most)), dim3(kThreads), 0,
                         stream, g);
    });
  });
  return launch_status();
}

extern "C" int64_t gq_rms_norm_backward_workspace(int64_t rows, int32_t H) {
  using namespace gq;
  if (rows < 0 || H < 1 || H > kNormMaxWidth) return -1;
  return most_back_groups(rows, H) * H * 4;
}

extern "C" int gq_rms_norm_backward(const void* d_y, int64_t d_y_stride, const void* h,
                                    int64_t h_stride, const void* d_h, int64_t d_h_stride,
                                    int32_t dtype, int64_t rows, int32_t H, const void* weight,
                                    int32_t weight_dtype, float eps, void* d_x, void* d_weight,
                                    void* workspace, int64_t workspace_bytes,
                                    hipStream_t stream) {
  using namespace gq;
  const int st = norm_checks(dtype, weight_dtype, rows, H, eps);
  if (st == kInvalid) return st;
  if (d_y_stride < H || h_stride < H || (d_h && d_h_stride < H)) return kInvalid;
  if (st != kOk) return st;
  if (rows == 0 && !d_weight) return kOk;
  if (rows > 0 && (!d_y || !h || !weight || !d_x)) return kInvalid;
  if (!element_aligned(d_y, dtype) || !element_aligned(h, dtype) || !element_aligned(d_h, dtype) ||
      !element_aligned(weight, weight_dtype) || !element_aligned(d_x, dtype) ||
      !element_aligned(d_weight, weight_dtype))
    return kInvalid;
  const int64_t groups = back_groups(rows, H);
  if (d_weight && rows > 0 &&
      (!workspace || !aligned16(workspace) || workspace_bytes < groups * H * 4))
    return kInvalid;
  if (!strides_fit(rows, d_y_stride) || !strides_fit(rows, h_stride) ||
      (d_h && !strides_fit(rows, d_h_stride)) || !strides_fit(rows, H))
    return kNotSupported;
  if (rows > 0 && (!apart(d_x, d_y, rows, d_y_stride, H) || !apart(d_x, h, rows, h_stride, H) ||
                   !apart(d_x, d_h, rows, d_h_stride, H)))
    return kInvalid;
  const int size = type_size(dtype);
  NormBackArgs g{static_cast<const char*>(d_y), static_cast<const char*>(h),
                 static_cast<const char*>(d_h), static_cast<const char*>(weight),
                 static_cast<char*>(d_x), d_weight ? static_cast<float*>(workspace) : nullptr,
                 rows, d_y_stride * size, h_stride * size, d_h_stride * size, H, eps};
  by_types(dtype, weight_dtype, [&](auto t, auto wt) {
    constexpr int T = decltype(t)::value, WT = decltype(wt)::value;
    if (rows > 0)
      by_row(rows, H, [&](auto w, auto c) {
        constexpr int kWaves = decltype(w)::value;
        hipLaunchKernelGGL((rms_norm_backward_kernel<T, WT, kWaves, decltype(c)::value>),
                           dim3((unsigned)groups), dim3(kNormThreads<kWaves>), 0, stream, g);
      });
    if (d_weight)
      hipLaunchKernelGGL((rms_norm_gain_kernel<WT>), dim3((unsigned)ceil_div64(H, kGainCols)),
                         dim3(kGainCols * kGainRuns), 0, stream, g.partial, (int)groups, H,
                         static_cast<char*>(d_weight));
  });
  return launch_status();
}
