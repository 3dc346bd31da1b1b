// Norms with the position rotation in the same pass, and the write of a step's rows into the caches.
//
//   n = x | x / sqrt(mean x^2 + eps) w | (x - mean x) / sqrt(var x + eps) w + b      (one head row of D dims)
//   (u, v) -> (u c - v s, v c + u s),  c = mul cos(pos f_i), s = mul sin(pos f_i)     (pairs of dims [off, off + R))
//
// The angle pos f_i is formed and reduced modulo 2 pi in 64 bits: a 32-bit angle at position 10^7 is off by half a
// radian.  What is left, |r| <= pi, goes through sincosf in 32 bits.  Norm statistics are 32-bit sums over the row's
// registers (the layer norm's variance from the centred values), and each result is rounded once.
//
// Both kernels move bytes: 16-byte loads and stores, one row per group of lanes, so a row's sums are shuffles.  The
// cos / sin table of a block's tokens is formed once in shared memory and serves all heads.
#include <cuda_fp8.h>

#include <cmath>

#include "lsa_common.cuh"
#include "sm100.cuh"

namespace lsa {
namespace {

__device__ int g_append_check;  // set when a slot was outside [-1, n_slots) (the row was skipped)

constexpr int NR_THREADS = 256;
constexpr int NR_TABLE = 8192;  // most rotary dims x tokens of one block's table (32 KB)

__device__ __forceinline__ float2 rope_cs(int64_t pos, double f, float mul) {
  const double a = static_cast<double>(pos) * f;
  const double n = rint(a * 0.15915494309189535);  // a / (2 pi)
  // 2 pi as a sum of two doubles
  const double r = fma(-n, 2.4492935982947064e-16, fma(-n, 6.2831853071795862, a));
  float s, c;
  sincosf(static_cast<float>(r), &s, &c);
  return make_float2(c * mul, s * mul);
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t u[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
// e4m3 codes of f / scale (the quotient itself, not a product with a reciprocal: a code is the nearest to it)
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale) {
  uint32_t u[2];
  #pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] / scale, f[4 * i + 1] / scale), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] / scale, f[4 * i + 3] / scale),
                                                 __NV_SATFINITE, __NV_E4M3);
    u[i] = lo | (hi << 16);
  }
  return make_uint2(u[0], u[1]);
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int G>
__device__ __forceinline__ float group_max(float v) {
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct NormRopeArgs {
  const uint16_t* x;
  int64_t ldt, ldh;  // element strides of x
  void* y;
  int64_t yldt, yldh;  // element strides of y
  float* scale;        // [T, H] (e4m3)
  const int64_t* pos;
  const double* freqs;  // [R / 2], or NULL: no rotation
  const float* weight;
  const float* bias;
  int64_t T;
  int H, D, norm, off, R, half;
  float eps, mul;
  int NT, HB;      // tokens and heads of a block
  int only_rotary;  // y is x and there is no norm: the other dims stay as they are
};

// A group of G lanes holds one head row, ITER 16-byte chunks a lane (chunk = lane + G * iter).  A block covers NT
// tokens x HB heads; the next row's loads are in flight while a row is computed.
template <int G, int ITER, bool FP8>
__global__ void __launch_bounds__(NR_THREADS) k_norm_rope(const NormRopeArgs a) {
  extern __shared__ float2 cs[];  // [NT][R / 2] cos, sin
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  constexpr int SLOTS = NR_THREADS / G;
  const int slot = threadIdx.x / G, gl = threadIdx.x % G, lane = threadIdx.x & 31;
  const int hsplit = (a.H + a.HB - 1) / a.HB;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / hsplit) * a.NT;
  const int h0 = static_cast<int>(blockIdx.x % hsplit) * a.HB;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.NT), a.T - t0)), nh = min(a.HB, a.H - h0);
  const int rows = nt * nh, chunks = a.D >> 3;
  const int c_lo = a.off >> 3, half_r = a.R >> 1, c_n = a.R >> 3;  // rotary chunks [c_lo, c_lo + c_n)

  bool mine[ITER];
  #pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = gl + G * i;
    mine[i] = c < chunks && (!a.only_rotary || (c >= c_lo && c < c_lo + c_n));
  }
  auto load = [&](int row, uint4 (&v)[ITER]) {
    const int t = row / nh, h = row - t * nh;
    const uint16_t* p = a.x + (t0 + t) * a.ldt + (h0 + h) * a.ldh;
    #pragma unroll
    for (int i = 0; i < ITER; ++i)
      v[i] = (row < rows && mine[i]) ? *reinterpret_cast<const uint4*>(p + 8 * (gl + G * i)) : make_uint4(0, 0, 0, 0);
  };
  uint4 nxt[ITER];
  load(slot, nxt);
  float w[ITER][8], b[ITER][8];
  #pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int c = gl + G * i;
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[i][j] = a.weight && c < chunks ? a.weight[8 * c + j] : 1.f;
      b[i][j] = a.bias && c < chunks ? a.bias[8 * c + j] : 0.f;
    }
  }
  if (a.freqs) {
    for (int i = threadIdx.x; i < nt * half_r; i += NR_THREADS) {
      const int t = i / half_r;
      cs[i] = rope_cs(a.pos[t0 + t], a.freqs[i - t * half_r], a.mul);
    }
    __syncthreads();
  }
  for (int base = 0; base < rows; base += SLOTS) {  // uniform over the block: the shuffles need every lane
    const int row = base + slot;
    float f[ITER][8];
    #pragma unroll
    for (int i = 0; i < ITER; ++i) unpack8(nxt[i], f[i]);
    if (base + SLOTS < rows) load(row + SLOTS, nxt);
    const float d = static_cast<float>(a.D);
    if (a.norm == LSA_NORM_LAYER) {
      float s = 0.f;
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) s += f[i][j];
      const float mean = group_sum<G>(s) / d;  // a division: the mean of a constant row is exact
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = mine[i] ? f[i][j] - mean : 0.f;  // chunks past D stay out of the sums
    }
    if (a.norm != LSA_NORM_NONE) {
      float s = 0.f;
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) s += f[i][j] * f[i][j];
      const float r = 1.f / sqrtf(group_sum<G>(s) / d + a.eps);
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * r * w[i][j] + b[i][j];
    }
    const int t = min(row, rows - 1) / nh;
    if (a.freqs) {
      const float2* tab = cs + t * half_r;
      if (a.half) {
        // pairs (i, i + R/2): the partner chunk is R/16 chunks away, in another lane (and iteration)
        const int hc = a.R >> 4;
        float g[ITER][8];
        #pragma unroll
        for (int i = 0; i < ITER; ++i) {
          const int rel = gl + G * i - c_lo;
          const int cp = min(max(rel < hc ? rel + hc : rel - hc, 0), c_n - 1) + c_lo;
          const int src = (lane & ~(G - 1)) | (cp & (G - 1)), it = cp / G;
          #pragma unroll
          for (int k = 0; k < ITER; ++k)
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float o = __shfl_sync(0xffffffffu, f[k][j], src);
              if (k == 0 || k == it) g[i][j] = o;
            }
        }
        #pragma unroll
        for (int i = 0; i < ITER; ++i) {
          const int rel = gl + G * i - c_lo;
          if (rel >= 0 && rel < c_n) {
            const bool first = rel < hc;
            #pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 e = tab[8 * (first ? rel : rel - hc) + j];
              f[i][j] = f[i][j] * e.x + (first ? -g[i][j] : g[i][j]) * e.y;
            }
          }
        }
      } else {
        #pragma unroll
        for (int i = 0; i < ITER; ++i) {
          const int rel = gl + G * i - c_lo;
          if (rel >= 0 && rel < c_n) {
            #pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 e = tab[4 * rel + j];
              const float u = f[i][2 * j], v = f[i][2 * j + 1];
              f[i][2 * j] = u * e.x - v * e.y;
              f[i][2 * j + 1] = v * e.x + u * e.y;
            }
          }
        }
      }
    }
    const int h = min(row, rows - 1) - t * nh;
    const int64_t o = (t0 + t) * a.yldt + (h0 + h) * a.yldh;
    if (FP8) {
      float m = 0.f;
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, mine[i] ? fabsf(f[i][j]) : 0.f);
      m = group_max<G>(m);
      const float sc = m > 0.f ? m / 448.f : 1.f;
      if (row < rows) {
        #pragma unroll
        for (int i = 0; i < ITER; ++i)
          if (mine[i])
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.y) + o + 8 * (gl + G * i)) = codes8(f[i], sc);
        if (gl == 0) a.scale[(t0 + t) * a.H + h0 + h] = sc;
      }
    } else if (row < rows) {
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        if (mine[i])
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.y) + o + 8 * (gl + G * i)) = pack8(f[i]);
    }
  }
}

template <int G, int ITER>
cudaError_t go_norm_rope(const NormRopeArgs& a, bool fp8, unsigned grid, size_t smem, cudaStream_t s) {
  return fp8 ? launch_pdl(k_norm_rope<G, ITER, true>, dim3(grid), dim3(NR_THREADS), smem, s, 0u, a)
             : launch_pdl(k_norm_rope<G, ITER, false>, dim3(grid), dim3(NR_THREADS), smem, s, 0u, a);
}

struct AppendArgs {
  const uint16_t* a;  // [T, 576]
  int64_t lda;
  const float* a_weight;  // [512], or NULL: no norm
  const uint16_t* k;      // [T, d_I], or NULL
  int64_t ldk;
  const float* k_weight;
  const float* k_bias;
  const int64_t* pos;
  const int64_t* slot;
  const double* freqs;  // [32], or NULL: no rotation
  uint16_t* kv;         // [n_slots, 576]
  void* kc;             // [n_slots, d_I]
  float* k_scale;       // [n_slots] (e4m3)
  int64_t T, n_slots;
  int d_I, k_norm, k_off, half, k_half;  // k_off < 0: index keys are not rotated
  float a_eps, k_eps, mul;
};

// One warp a latent row (chunks lane, lane + 32 are the 512 normed dims, chunk 64 + lane of the first 8 lanes the
// rotary ones), another warp its index key.  Lane i forms cos and sin of pair i; the lanes that rotate fetch theirs by
// shuffles, so there is no shared memory and no barrier on the way.
template <bool KEYS, bool FP8>
__global__ void __launch_bounds__(128) k_cache_append(const AppendArgs a) {
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = KEYS ? static_cast<int64_t>(blockIdx.x) * 2 + (warp >> 1) : static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (t >= a.T) return;
  const bool is_key = KEYS && (warp & 1);
  const int64_t slot = a.slot[t];
  const int64_t pos = a.freqs ? a.pos[t] : 0;
  const double fr = a.freqs ? a.freqs[lane] : 0.0;
  if (!is_key) {
    const uint16_t* p = a.a + t * a.lda;
    uint4 v[3];
    v[0] = *reinterpret_cast<const uint4*>(p + 8 * lane);
    v[1] = *reinterpret_cast<const uint4*>(p + 8 * (lane + 32));
    v[2] = lane < 8 ? *reinterpret_cast<const uint4*>(p + 8 * (lane + 64)) : make_uint4(0, 0, 0, 0);
    float f[3][8];
    #pragma unroll
    for (int i = 0; i < 3; ++i) unpack8(v[i], f[i]);
    if (a.a_weight) {
      float w[2][8];
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = a.a_weight[8 * (lane + 32 * i) + j];
      float s = 0.f;
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) s += f[i][j] * f[i][j];
      const float r = 1.f / sqrtf(warp_sum(s) * (1.f / 512.f) + a.a_eps);
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) f[i][j] = f[i][j] * r * w[i][j];
    }
    if (a.freqs) {
      const float2 e = rope_cs(pos, fr, a.mul);
      if (a.half) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float g = __shfl_xor_sync(0xffffffffu, f[2][j], 4);
          const int pair = 8 * (lane & 3) + j;
          const float c = __shfl_sync(0xffffffffu, e.x, pair), s = __shfl_sync(0xffffffffu, e.y, pair);
          f[2][j] = f[2][j] * c + ((lane & 4) ? g : -g) * s;
        }
      } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pair = (4 * lane + j) & 31;
          const float c = __shfl_sync(0xffffffffu, e.x, pair), s = __shfl_sync(0xffffffffu, e.y, pair);
          const float u = f[2][2 * j], w = f[2][2 * j + 1];
          f[2][2 * j] = u * c - w * s;
          f[2][2 * j + 1] = w * c + u * s;
        }
      }
    }
    if (slot < 0 || slot >= a.n_slots) {
      if (slot != -1 && lane == 0) atomicExch(&g_append_check, 1);
      return;
    }
    uint16_t* o = a.kv + slot * 576;
    *reinterpret_cast<uint4*>(o + 8 * lane) = pack8(f[0]);
    *reinterpret_cast<uint4*>(o + 8 * (lane + 32)) = pack8(f[1]);
    if (lane < 8) *reinterpret_cast<uint4*>(o + 8 * (lane + 64)) = pack8(f[2]);
  } else {
    const int chunks = a.d_I >> 3;
    const bool mine = lane < chunks;
    float f[8];
    unpack8(mine ? *reinterpret_cast<const uint4*>(a.k + t * a.ldk + 8 * lane) : make_uint4(0, 0, 0, 0), f);
    const float d = static_cast<float>(a.d_I);
    if (a.k_norm == LSA_NORM_LAYER) {
      float s = 0.f;
      #pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j];
      const float mean = warp_sum(s) / d;
      #pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = mine ? f[j] - mean : 0.f;
    }
    if (a.k_norm != LSA_NORM_NONE) {
      float s = 0.f;
      #pragma unroll
      for (int j = 0; j < 8; ++j) s += f[j] * f[j];
      const float r = 1.f / sqrtf(warp_sum(s) / d + a.k_eps);
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float w = a.k_weight && mine ? a.k_weight[8 * lane + j] : 1.f;
        const float b = a.k_bias && mine ? a.k_bias[8 * lane + j] : 0.f;
        f[j] = f[j] * r * w + b;
      }
    }
    if (a.freqs && a.k_off >= 0) {
      const float2 e = rope_cs(pos, fr, a.mul);
      const int rel = lane - (a.k_off >> 3);
      const bool rot = rel >= 0 && rel < 8;
      if (a.k_half) {
        #pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float g = __shfl_sync(0xffffffffu, f[j], (rel < 4 ? lane + 4 : lane - 4) & 31);
          const int pair = 8 * (rel & 3) + j;
          const float c = __shfl_sync(0xffffffffu, e.x, pair), s = __shfl_sync(0xffffffffu, e.y, pair);
          if (rot) f[j] = f[j] * c + (rel < 4 ? -g : g) * s;
        }
      } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pair = (4 * rel + j) & 31;
          const float c = __shfl_sync(0xffffffffu, e.x, pair), s = __shfl_sync(0xffffffffu, e.y, pair);
          const float u = f[2 * j], w = f[2 * j + 1];
          if (rot) {
            f[2 * j] = u * c - w * s;
            f[2 * j + 1] = w * c + u * s;
          }
        }
      }
    }
    if (FP8) {
      float m = 0.f;
      #pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, mine ? fabsf(f[j]) : 0.f);
      m = warp_max(m);
      const float sc = m > 0.f ? m / 448.f : 1.f;
      if (slot < 0 || slot >= a.n_slots) return;
      if (mine)
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.kc) + slot * a.d_I + 8 * lane) = codes8(f, sc);
      if (lane == 0) a.k_scale[slot] = sc;
    } else {
      if (slot < 0 || slot >= a.n_slots) return;
      if (mine) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.kc) + slot * a.d_I + 8 * lane) = pack8(f);
    }
  }
}

}  // namespace

int sm_count();

int launch_norm_rope(const void* x, int64_t ldt, int64_t ldh, int64_t T, int H, int D, int norm, const float* weight,
                     const float* bias, float eps, const double* freqs, int off, int R, int layout, float mul,
                     const int64_t* pos, void* y, int64_t yldt, int64_t yldh, int dtype, float* scale,
                     cudaStream_t s) {
  NormRopeArgs a;
  a.x = static_cast<const uint16_t*>(x);
  a.ldt = ldt;
  a.ldh = ldh;
  a.y = y;
  a.yldt = yldt;
  a.yldh = yldh;
  a.scale = scale;
  a.pos = pos;
  a.freqs = freqs;
  a.weight = weight;
  a.bias = bias;
  a.T = T;
  a.H = H;
  a.D = D;
  a.norm = norm;
  a.off = off;
  a.R = freqs ? R : 0;
  a.half = layout == LSA_ROPE_HALF;
  a.eps = eps;
  a.mul = mul;
  const bool fp8 = dtype == LSA_FP8_E4M3;
  a.only_rotary = !fp8 && norm == LSA_NORM_NONE && x == y && ldt == yldt && ldh == yldh;
  // lanes a row: its 16-byte chunks spread over a power of two of lanes, with one or three chunks a lane where that
  // leaves none idle, else a whole warp
  const int n = D >> 3;
  int G = 32, it = (n + 31) / 32;
  for (int g = 4; g <= 16; g *= 2)
    if (n == g || n == 3 * g) {
      G = g;
      it = n / g;
    }
  if (n < 4) {
    G = 4;
    it = 1;
  }
  // a block's rows: four to a group of lanes when there are many rows (more loads in flight for each pass through the
  // table), one when the whole call would not fill the GPU's 8 blocks an SM
  const int slots = NR_THREADS / G;
  const int64_t total = T * H;
  const int64_t want = total > static_cast<int64_t>(sm_count()) * 8 * slots * 2 ? 4 * slots : slots;
  if (H >= want) {
    a.NT = 1;
    a.HB = static_cast<int>(want);
  } else {
    a.HB = H;
    a.NT = static_cast<int>(want / H);
    if (a.R > 0 && a.NT > NR_TABLE / a.R) a.NT = NR_TABLE / a.R;
    if (a.NT < 1) a.NT = 1;
  }
  const int64_t grid = cdiv(T, a.NT) * cdiv(H, a.HB);
  if (grid > 0x7FFFFFFF) return LSA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(a.NT) * (a.R / 2) * sizeof(float2);
  const unsigned g = static_cast<unsigned>(grid);
  cudaError_t e = cudaErrorInvalidValue;
  if (G == 4) e = it == 1 ? go_norm_rope<4, 1>(a, fp8, g, smem, s) : go_norm_rope<4, 3>(a, fp8, g, smem, s);
  else if (G == 8) e = it == 1 ? go_norm_rope<8, 1>(a, fp8, g, smem, s) : go_norm_rope<8, 3>(a, fp8, g, smem, s);
  else if (G == 16) e = it == 1 ? go_norm_rope<16, 1>(a, fp8, g, smem, s) : go_norm_rope<16, 3>(a, fp8, g, smem, s);
  else if (it == 1) e = go_norm_rope<32, 1>(a, fp8, g, smem, s);
  else if (it == 2) e = go_norm_rope<32, 2>(a, fp8, g, smem, s);
  else if (it == 3) e = go_norm_rope<32, 3>(a, fp8, g, smem, s);
  else if (it == 4) e = go_norm_rope<32, 4>(a, fp8, g, smem, s);
  return cuda_status(e);
}

int launch_cache_append(const void* x, int64_t ldx, const float* x_weight, float x_eps, const void* k, int64_t ldk,
                        int d_I, int k_norm, const float* k_weight, const float* k_bias, float k_eps, int k_off,
                        int k_layout, const double* freqs, int layout, float mul, const int64_t* pos,
                        const int64_t* slot, int64_t T, void* kv, int64_t n_slots, void* kc, int k_dtype,
                        float* k_scale, cudaStream_t s) {
  AppendArgs a;
  a.a = static_cast<const uint16_t*>(x);
  a.lda = ldx;
  a.a_weight = x_weight;
  a.k = static_cast<const uint16_t*>(k);
  a.ldk = ldk;
  a.k_weight = k_weight;
  a.k_bias = k_bias;
  a.pos = pos;
  a.slot = slot;
  a.freqs = freqs;
  a.kv = static_cast<uint16_t*>(kv);
  a.kc = kc;
  a.k_scale = k_scale;
  a.T = T;
  a.n_slots = n_slots;
  a.d_I = d_I;
  a.k_norm = k_norm;
  a.k_off = k_off;
  a.half = layout == LSA_ROPE_HALF;
  a.k_half = k_layout == LSA_ROPE_HALF;
  a.a_eps = x_eps;
  a.k_eps = k_eps;
  a.mul = mul;
  const int64_t grid = cdiv(T, k ? 2 : 4);
  if (grid > 0x7FFFFFFF) return LSA_ERR_UNSUPPORTED;
  const dim3 g(static_cast<unsigned>(grid)), b(128);
  if (!k) return cuda_status(launch_pdl(k_cache_append<false, false>, g, b, 0, s, 0u, a));
  if (k_dtype == LSA_FP8_E4M3) return cuda_status(launch_pdl(k_cache_append<true, true>, g, b, 0, s, 0u, a));
  return cuda_status(launch_pdl(k_cache_append<true, false>, g, b, 0, s, 0u, a));
}

// Angular frequencies base^(-2i/R), scaled for long contexts.  YaRN (arXiv 2309.00071, section 3.2): dims that turn
// more than beta_fast times over the original length keep their frequency, those that turn less than beta_slow times
// are divided by the factor, with a linear ramp between; cos and sin are multiplied by 0.1 ln(factor) + 1.
void rope_freqs(int R, double base, int scaling, double factor, int64_t original_len, double beta_fast,
                double beta_slow, double* freqs, float* mul) {
  const double two_pi = 6.283185307179586;
  double low = 0, high = 0;
  if (scaling == LSA_ROPE_YARN) {
    auto dim = [&](double beta) { return R * std::log(original_len / (beta * two_pi)) / (2 * std::log(base)); };
    low = std::fmax(std::floor(dim(beta_fast)), 0.0);
    high = std::fmin(std::ceil(dim(beta_slow)), R - 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / R);
    double r = scaling == LSA_ROPE_LINEAR ? 1.0 : 0.0;  // the share of the divided frequency
    if (scaling == LSA_ROPE_YARN) r = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0.0), 1.0);
    freqs[i] = (1.0 - r) * f + r * f / factor;
  }
  *mul = scaling == LSA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
}

// device check of the cache append, read and cleared; -1: CUDA error
int take_append_check() {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_append_check, sizeof(int)) != cudaSuccess) return -1;
  const int zero = 0;
  if (v != 0 && cudaMemcpyToSymbol(g_append_check, &zero, sizeof(int)) != cudaSuccess) return -1;
  return v;
}

}  // namespace lsa
