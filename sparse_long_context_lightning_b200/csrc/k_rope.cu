// Norms with the position rotation in the same pass, and the write of a step's rows into the caches.
//
//   n = x | x / sqrt(mean x^2 + eps) w | (x - mean x) / sqrt(var x + eps) w + b      (one head row of D dims)
//   (u, v) -> (u c - v s, v c + u s),  c = mul cos(pos f_i), s = mul sin(pos f_i)     (pairs of dims [off, off + R))
//
// The angle pos f_i is formed and reduced to a part of a turn in 64 bits: a 32-bit angle at position 10^7 is off by half
// a radian.  What is left, half a turn at most, goes through sincospif in 32 bits.  Norm statistics are 32-bit sums over
// the row's registers (the layer norm's variance from the centred values), and each result is rounded once.
//
// Both kernels move bytes (16-byte loads and stores; a row's sums are shuffles among the lanes that hold it), and both
// were bound by their instructions first: no division and no 64-bit product is left in the loop over rows.
#include <cuda_fp8.h>

#include <cmath>

#include "lsa_common.cuh"
#include "sm100.cuh"

namespace lsa {
namespace {

__device__ int g_append_check;  // set when a slot was outside [-1, n_slots) (the row was skipped)

constexpr int NR_THREADS = 128;

__device__ __forceinline__ float2 rope_cs(int64_t pos, double f, float mul) {
  const double t = static_cast<double>(pos) * f * 0.15915494309189535;  // turns
  float s, c;
  sincospif(2.f * static_cast<float>(t - rint(t)), &s, &c);
  return make_float2(c * mul, s * mul);
}

__device__ __forceinline__ float lo_f(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_f(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = lo_f(u[i]);
    f[2 * i + 1] = hi_f(u[i]);
  }
}
// eight results, rounded to bf16 (the caches' and queries' type)
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y));
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
// The larger of two, NaN if either is: a NaN has to reach the row's scale, since the indexer's ReLU takes a NaN product of
// codes for 0 and only the scale then carries it into the score.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The row's scale and its reciprocal (0 where that would overflow, and for an infinite or NaN scale).  Codes are formed from value * reciprocal: a quotient
// takes ten instructions an element, and the product, off by two roundings of 32 bits, can only choose another code for a
// value within 2^-22 of the border of two, where the norm's own rounding chooses as much.
__device__ __forceinline__ float2 row_scale(float amax) {
  const float s = amax == 0.f ? 1.f : amax * (1.f / 448.f);
  return make_float2(s, s > 1e-35f ? __fdividef(1.f, s) : 0.f);
}
// s / d, off by less than a rounding: the mean of a constant row is that constant (s = c d is exact for a bf16 c)
__device__ __forceinline__ float mean_of(float s, float d, float inv_d) {
  const float q = s * inv_d;
  return fmaf(fmaf(-q, d, s), inv_d, q);
}
// two 32-bit operations an instruction
__device__ __forceinline__ uint64_t bits(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 floats(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return floats(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
  return floats(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return floats(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

__device__ __forceinline__ uint32_t codes2(float2 v, float2 inv) {
  const float2 q = mul2(v, inv);
  uint16_t u;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(q.y), "f"(q.x));
  return u;
}
// the values over the scale where there is no reciprocal: codes are then formed with 1
template <int N>
__device__ __forceinline__ float tiny_row(float2 (&f)[N], const float2& sc) {
  if (sc.y != 0.f) return sc.y;
  #pragma unroll
  for (int i = 0; i < N; ++i) f[i] = make_float2(f[i].x / sc.x, f[i].y / sc.x);
  return 1.f;
}
__device__ __forceinline__ uint2 codes8(const float2 (&f)[4], float2 inv) {
  return make_uint2(codes2(f[0], inv) | (codes2(f[1], inv) << 16), codes2(f[2], inv) | (codes2(f[3], inv) << 16));
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
  for (int o = G / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
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
  int H, D, off, R, half;
  float eps, mul;
  int spt_log, HB, TB;  // a block: 2^spt_log row slots a token, HB heads, TB times (slots / 2^spt_log) tokens
  int only_rotary;  // y is x and there is no norm: the other dims stay as they are
};

// A group of G lanes holds a head row, ITER 16-byte chunks a lane.  The rotary chunks come first: lane p holds chunk p
// and its partner R / 16 chunks on, the two halves of eight (i, i + R/2) pairs, in two neighbouring iterations, so that
// neither layout moves a value between lanes; the other chunks fill the rest.  A block forms one table of cos and sin
// for its tokens (the chain of loads, 64-bit products and sincospif takes longer than 64 rows) and walks their heads, RPT
// rows a slot at a time, with the next rows' loads in flight; weights and table lie in shared memory, because 32 registers
// of weights halve the warps of an SM (70 us against 45 for 8192 x 64 rows of 128 dims).  Products and sums go two an
// instruction.  Small blocks (128 threads, six an SM) wait for each other least: 43.4 us against 44.6 at 256 threads and
// 70 at 512; a grid of resident blocks with two tables in turn took 55.  Six blocks leave a thread 80 registers, at which
// two chunks a lane spill 4 to 16 bytes: for bf16 that costs less than a block (8192 x 64 rows of 128, RMS norm: 43.0 us
// against 44.6 at five), for codes, which also hold a row's scale (4 to 60 bytes; at most 12 at five), it costs more (4099 x 64 rows of 128,
// layer norm: 28.7 us against 27.3 at five; RMS norm 25.5 against 24.2).
// 8192 x 64 rows of 128 dims, RMS norm, whole heads rotated: 45.9 us, 5850 GB/s.  2047 x 128 rows of 64, no norm, into
// their place in rows of 1152 bytes: 15.9 us, 4210 GB/s; neither HBM (28% of its peak) nor the issue slots (34%) are full:
// it waits for its loads, and its 1024 blocks are little more than the 888 that fit at a time (11.4 us in the L2).
// 4099 x 64 rows of 128, layer norm, to codes: 27.9 us, 3650 GB/s: about 18 instructions an element (three reductions and a
// scale a row), 55% of the issue slots at 20 warps an SM; what stalls it is the shuffles and the table in shared memory.
template <int G, int ITER, int NORM, bool FP8>
__global__ void __launch_bounds__(NR_THREADS, ITER <= 2 ? (FP8 ? 5 : 6) : 4) k_norm_rope(const NormRopeArgs a) {
  extern __shared__ __align__(16) float2 cs[];  // [tokens][R / 2] cos, sin | weight [D] | bias [D]
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  constexpr int RPT = ITER <= 2 ? 2 : 1;
  const int slot = threadIdx.x / G, gl = threadIdx.x % G;
  const int spt = 1 << a.spt_log, NT = (NR_THREADS / G) >> a.spt_log;
  const int tk = slot >> a.spt_log, hs = slot & (spt - 1);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * NT * a.TB;
  const int nt = static_cast<int>(min(static_cast<int64_t>(NT) * a.TB, a.T - t0));  // tokens of this block
  const int half_r = a.R >> 1;
  const int h_first = static_cast<int>(blockIdx.y) * a.HB + hs;
  const int h_end = min(a.H, static_cast<int>(blockIdx.y + 1) * a.HB);

  // the lane's chunks
  int off[ITER];  // element offset, or -1
  bool rot[(ITER + 1) / 2];
  {
    const int P = a.R >> 4, c_lo = a.off >> 3, n_rest = a.only_rotary ? 0 : (a.D >> 3) - 2 * P;
    int base = 0;
    #pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int pj = i + (1 - i % 2) < ITER ? min(max(P - G * (i / 2), 0), G) : 0;  // a last odd iteration holds no pair
      if (i % 2 == 0) rot[i / 2] = gl < pj;
      int c = c_lo + (i % 2) * P + G * (i / 2) + gl;
      if (gl >= pj) {
        const int e = base + gl - pj;
        c = e >= n_rest ? -1 : e < c_lo || P == 0 ? e : e + 2 * P;
      }
      base += G - pj;
      off[i] = c < 0 ? -1 : 8 * c;
    }
  }
  // rows k of the slot's next step: token tl, heads h_first + lh + k spt
  uint4 v[RPT][ITER];
  int tl = tk, lh = 0;
  const int64_t xstep = spt * a.ldh, ystep = spt * a.yldh;
  const int64_t xturn = NT * a.ldt - a.HB * a.ldh, yturn = NT * a.yldt - a.HB * a.yldh;  // from a token's end to the next
  const uint16_t* px = a.x + (t0 + tk) * a.ldt + h_first * a.ldh;
  auto load = [&]() {
    #pragma unroll
    for (int k = 0; k < RPT; ++k) {
      const bool live = tl < nt && h_first + lh + k * spt < h_end;
      #pragma unroll
      for (int i = 0; i < ITER; ++i)
        v[k][i] = live && off[i] >= 0 ? *reinterpret_cast<const uint4*>(px + off[i]) : make_uint4(0, 0, 0, 0);
      if (k == 0 || lh + spt < a.HB) px += xstep;
    }
    lh += RPT * spt;
    if (lh >= a.HB) {
      lh = 0;
      tl += NT;
      px += xturn;
    }
  };
  load();
  // Entries of four floats (two pairs; four weights) that the lanes of a row read together lie side by side.
  float* w_s = reinterpret_cast<float*>(cs + static_cast<size_t>(NT) * a.TB * half_r);
  float* b_s = w_s + a.D;
  const int P = a.R >> 4;
  float* cf = reinterpret_cast<float*>(cs);
  auto put = [&](int q, int p, float2 v) {  // token q, pair p: an entry is cos of two pairs, then sin
    const int e = a.half ? ((p & 7) >> 1) * P + (p >> 3) : ((p & 3) >> 1) * 2 * P + (p >> 2);
    float* o = cf + 2 * q * half_r + 4 * e + (p & 1);
    o[0] = v.x;
    o[2] = v.y;
  };
  auto weight_at = [&](int i) { return 4 * (((i & 7) >> 2) * (a.D >> 3) + (i >> 3)) + (i & 3); };
  {
    // the first of each thread's loads go out together
    const int i0 = threadIdx.x, q0 = half_r ? i0 / half_r : 0;
    const bool any = i0 < nt * half_r, wany = NORM != LSA_NORM_NONE && i0 < a.D;
    const int64_t pos = any ? a.pos[t0 + q0] : 0;
    const double fr = any ? a.freqs[i0 - q0 * half_r] : 0.0;
    const float w0 = wany && a.weight ? a.weight[i0] : 1.f, b0 = wany && a.bias ? a.bias[i0] : 0.f;
    if (any) put(q0, i0 - q0 * half_r, rope_cs(pos, fr, a.mul));
    if (wany) {
      w_s[weight_at(i0)] = w0;
      if (NORM == LSA_NORM_LAYER) b_s[weight_at(i0)] = b0;
    }
    for (int i = i0 + NR_THREADS; i < nt * half_r; i += NR_THREADS) {
      const int q = i / half_r;
      put(q, i - q * half_r, rope_cs(a.pos[t0 + q], a.freqs[i - q * half_r], a.mul));
    }
    if (NORM != LSA_NORM_NONE)
      for (int i = i0 + NR_THREADS; i < a.D; i += NR_THREADS) {
        w_s[weight_at(i)] = a.weight ? a.weight[i] : 1.f;
        if (NORM == LSA_NORM_LAYER) b_s[weight_at(i)] = a.bias ? a.bias[i] : 0.f;
      }
  }
  __syncthreads();
  const float d = static_cast<float>(a.D), inv_d = 1.f / d;
  int64_t yo = (t0 + tk) * a.yldt + h_first * a.yldh;
  float* ps = FP8 ? a.scale + (t0 + tk) * a.H + h_first : nullptr;
  for (int tb = 0; tb < a.TB && NT * tb < nt; ++tb) {  // uniform over the block: the shuffles need every lane
    const int tq = NT * tb + tk;
    const float4* tab = reinterpret_cast<const float4*>(cs + min(tq, nt - 1) * half_r);  // two pairs an entry
    for (int hb = 0; hb < a.HB; hb += RPT * spt) {
      const int h = h_first + hb, rows = hb + spt < a.HB ? RPT : 1;
      float2 f[RPT][ITER][4];
      #pragma unroll
      for (int k = 0; k < RPT; ++k)
        #pragma unroll
        for (int i = 0; i < ITER; ++i) {
          const uint32_t u[4] = {v[k][i].x, v[k][i].y, v[k][i].z, v[k][i].w};
          #pragma unroll
          for (int j = 0; j < 4; ++j) f[k][i][j] = make_float2(lo_f(u[j]), hi_f(u[j]));
        }
      load();
      if (NORM != LSA_NORM_NONE) {
        float r[RPT];
        #pragma unroll
        for (int k = 0; k < RPT; ++k) {
          if (NORM == LSA_NORM_LAYER) {
            float2 s = f[k][0][0];
            #pragma unroll
            for (int i = 0; i < ITER; ++i)
              #pragma unroll
              for (int j = 0; j < 4; ++j)
                if (i + j > 0) s = add2(s, f[k][i][j]);
            const float mean = mean_of(group_sum<G>(s.x + s.y), d, inv_d);
            #pragma unroll
            for (int i = 0; i < ITER; ++i) {
              const float2 mi = both(off[i] >= 0 ? -mean : 0.f);  // what is behind D stays out of the sums
              #pragma unroll
              for (int j = 0; j < 4; ++j) f[k][i][j] = add2(f[k][i][j], mi);
            }
          }
          float2 s = mul2(f[k][0][0], f[k][0][0]);
          #pragma unroll
          for (int i = 0; i < ITER; ++i)
            #pragma unroll
            for (int j = 0; j < 4; ++j)
              if (i + j > 0) s = fma2(f[k][i][j], f[k][i][j], s);
          r[k] = rsqrtf(group_sum<G>(s.x + s.y) * inv_d + a.eps);
        }
        #pragma unroll
        for (int i = 0; i < ITER; ++i) {
          const int o = max(off[i], 0) >> 3;
          #pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 w = *reinterpret_cast<const float4*>(w_s + 4 * (o + q * (a.D >> 3)));
            const float4 b = NORM == LSA_NORM_LAYER ? *reinterpret_cast<const float4*>(b_s + 4 * (o + q * (a.D >> 3)))
                                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            #pragma unroll
            for (int k = 0; k < RPT; ++k) {
              float2* g = f[k][i] + 2 * q;
              g[0] = mul2(g[0], both(r[k]));
              g[1] = mul2(g[1], both(r[k]));
              if (NORM == LSA_NORM_LAYER) {
                g[0] = fma2(g[0], make_float2(w.x, w.y), make_float2(b.x, b.y));
                g[1] = fma2(g[1], make_float2(w.z, w.w), make_float2(b.z, b.w));
              } else {
                g[0] = mul2(g[0], make_float2(w.x, w.y));
                g[1] = mul2(g[1], make_float2(w.z, w.w));
              }
            }
          }
        }
      }
      if (half_r) {
        #pragma unroll
        for (int q = 0; q < ITER / 2; ++q) {
          if (!rot[q]) continue;
          #pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (a.half) {
              const float4 z = tab[e * P + G * q + gl];  // cos of pairs 2e, 2e + 1 of the chunk, then sin
              const float2 c = make_float2(z.x, z.y), n = make_float2(z.z, z.w), m = make_float2(-z.z, -z.w);
              #pragma unroll
              for (int k = 0; k < RPT; ++k) {
                const float2 u = f[k][2 * q][e], g = f[k][2 * q + 1][e];
                f[k][2 * q][e] = fma2(g, m, mul2(u, c));
                f[k][2 * q + 1][e] = fma2(u, n, mul2(g, c));
              }
            } else {
              const int it = 2 * q + (e >> 1), j = 2 * (e & 1);
              const float4 z = tab[(e & 1) * 2 * P + G * q + gl + (e >> 1) * P];
              #pragma unroll
              for (int k = 0; k < RPT; ++k) {
                float2 u = f[k][it][j];
                f[k][it][j] = make_float2(u.x * z.x - u.y * z.z, u.y * z.x + u.x * z.z);
                u = f[k][it][j + 1];
                f[k][it][j + 1] = make_float2(u.x * z.y - u.y * z.w, u.y * z.y + u.x * z.w);
              }
            }
          }
        }
      }
      #pragma unroll
      for (int k = 0; k < RPT; ++k) {
        if (k >= rows) break;
        const bool live = tq < nt && h + k * spt < h_end;
        if (FP8) {
          float m = 0.f;
          #pragma unroll
          for (int i = 0; i < ITER; ++i) {
            float mi = 0.f;
            #pragma unroll
            for (int j = 0; j < 4; ++j) mi = max_nan(mi, max_nan(fabsf(f[k][i][j].x), fabsf(f[k][i][j].y)));
            m = max_nan(m, off[i] >= 0 ? mi : 0.f);
          }
          const float2 sc = row_scale(group_max<G>(m));
          float inv = sc.y;
          if (inv == 0.f) {
            #pragma unroll
            for (int i = 0; i < ITER; ++i) inv = tiny_row(f[k][i], sc);
          }
          if (live) {
            uint8_t* py = static_cast<uint8_t*>(a.y) + yo;
            #pragma unroll
            for (int i = 0; i < ITER; ++i)
              if (off[i] >= 0) *reinterpret_cast<uint2*>(py + off[i]) = codes8(f[k][i], both(inv));
            if (gl == 0) ps[k * spt] = sc.x;
          }
        } else if (live) {
          uint16_t* py = static_cast<uint16_t*>(a.y) + yo;
          #pragma unroll
          for (int i = 0; i < ITER; ++i)
            if (off[i] >= 0) *reinterpret_cast<uint4*>(py + off[i]) = pack8(f[k][i]);
        }
        yo += ystep;
      }
      if (FP8) ps += RPT * spt;
    }
    yo += yturn;
    if (FP8) ps += NT * a.H - (a.HB + RPT * spt - 1) / (RPT * spt) * (RPT * spt);
  }
}

template <int G, int ITER>
cudaError_t go_norm_rope(const NormRopeArgs& a, int norm, bool fp8, dim3 grid, size_t smem, cudaStream_t s) {
  const dim3 b(NR_THREADS);
  if (norm == LSA_NORM_NONE)
    return fp8 ? launch_pdl(k_norm_rope<G, ITER, LSA_NORM_NONE, true>, grid, b, smem, s, 0u, a)
               : launch_pdl(k_norm_rope<G, ITER, LSA_NORM_NONE, false>, grid, b, smem, s, 0u, a);
  if (norm == LSA_NORM_RMS)
    return fp8 ? launch_pdl(k_norm_rope<G, ITER, LSA_NORM_RMS, true>, grid, b, smem, s, 0u, a)
               : launch_pdl(k_norm_rope<G, ITER, LSA_NORM_RMS, false>, grid, b, smem, s, 0u, a);
  return fp8 ? launch_pdl(k_norm_rope<G, ITER, LSA_NORM_LAYER, true>, grid, b, smem, s, 0u, a)
             : launch_pdl(k_norm_rope<G, ITER, LSA_NORM_LAYER, false>, grid, b, smem, s, 0u, a);
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

// two bf16 of a row: neighbours, or `far` elements apart
__device__ __forceinline__ float2 load_pair(const uint16_t* p, int far) {
  if (far == 1) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(lo_f(u), hi_f(u));
  }
  return make_float2(bf16_bits_to_f32(p[0]), bf16_bits_to_f32(p[far]));
}
__device__ __forceinline__ void store_pair(uint16_t* p, int far, float2 v) {
  const uint32_t u = pack2(v.x, v.y);
  if (far == 1) {
    *reinterpret_cast<uint32_t*>(p) = u;
  } else {
    p[0] = static_cast<uint16_t>(u);
    p[far] = static_cast<uint16_t>(u >> 16);
  }
}
__device__ __forceinline__ void store_codes(uint8_t* p, int far, uint32_t u) {
  if (far == 1) {
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(u);
  } else {
    p[0] = static_cast<uint8_t>(u);
    p[far] = static_cast<uint8_t>(u >> 8);
  }
}

// A warp a latent row, another its index key.  Lane i of the first holds 16 of the 512 normed dims and pair i of the
// rotary ones; lane i of the second the key's pair i and up to four of its other dims: no value moves between lanes but
// the sums.  A step's few rows are bound by the chain of loads, sums and stores, a prompt's by the rows that an SM holds
// meanwhile, so registers are kept to 12 blocks an SM (the weights are read when they are used).  16 tokens: 1.9 us with
// warm caches, 3.4 us cold (2.9 warm with both rows in one warp); 8192 tokens with codes: 10.9 us cold, 2040 GB/s (12.0
// with 9 blocks an SM; inputs in turn 7.4 us, 7.7 with 10 blocks, whose 48 registers spare the 8 bytes that 40 spill).
template <bool KEYS, bool FP8>
__global__ void __launch_bounds__(128, 12) k_cache_append(const AppendArgs a) {
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = KEYS ? static_cast<int64_t>(blockIdx.x) * 2 + (warp >> 1) : static_cast<int64_t>(blockIdx.x) * 4 + warp;
  if (t >= a.T) return;
  const int64_t slot = a.slot[t];
  const int64_t pos = a.freqs ? a.pos[t] : 0;
  const double fr = a.freqs ? a.freqs[lane] : 0.0;
  const bool write = slot >= 0 && slot < a.n_slots;
  if (!KEYS || (warp & 1) == 0) {
    const uint16_t* p = a.a + t * a.lda;
    const uint4 v[2] = {*reinterpret_cast<const uint4*>(p + 8 * lane), *reinterpret_cast<const uint4*>(p + 8 * (lane + 32))};
    const int r_at = 512 + (a.half ? lane : 2 * lane), r_far = a.half ? 32 : 1;
    float2 r = load_pair(p + r_at, r_far);
    if (!write && slot != -1 && lane == 0) atomicExch(&g_append_check, 1);
    float f[2][8];
    unpack8(v[0], f[0]);
    unpack8(v[1], f[1]);
    if (a.a_weight) {
      float s = 0.f;
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(f[i][j], f[i][j], s);
      const float q = rsqrtf(warp_sum(s) * (1.f / 512.f) + a.a_eps);
      const bool wide = (reinterpret_cast<uintptr_t>(a.a_weight) & 15) == 0;
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* w = a.a_weight + 8 * (lane + 32 * i);
        #pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float4 g = wide ? *reinterpret_cast<const float4*>(w + 4 * p)
                                : make_float4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
          f[i][4 * p] = f[i][4 * p] * q * g.x;
          f[i][4 * p + 1] = f[i][4 * p + 1] * q * g.y;
          f[i][4 * p + 2] = f[i][4 * p + 2] * q * g.z;
          f[i][4 * p + 3] = f[i][4 * p + 3] * q * g.w;
        }
      }
    }
    if (a.freqs) {
      const float2 cs = rope_cs(pos, fr, a.mul);
      r = make_float2(r.x * cs.x - r.y * cs.y, r.y * cs.x + r.x * cs.y);
    }
    if (write) {
      uint16_t* o = a.kv + slot * 576;
      *reinterpret_cast<uint4*>(o + 8 * lane) = pack8(f[0]);
      *reinterpret_cast<uint4*>(o + 8 * (lane + 32)) = pack8(f[1]);
      store_pair(o + r_at, r_far, r);
    }
  } else {
    // the key's rotary pair, and dims 2 lane, 2 lane + 1 and 64 further of the others
    const bool turn = a.k_off >= 0;
    const int others = a.d_I - (turn ? 64 : 0);
    const int k_at = turn ? a.k_off + (a.k_half ? lane : 2 * lane) : 0, k_far = a.k_half ? 32 : 1;
    const uint16_t* kp = a.k + t * a.ldk;
    int at[3], far[3] = {k_far, 1, 1};
    float2 v[3], w[3], b[3];
    at[0] = turn ? k_at : -1;
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * lane + 64 * j;
      at[j + 1] = e >= others ? -1 : turn && e >= a.k_off ? e + 64 : e;
    }
    #pragma unroll
    for (int j = 0; j < 3; ++j) {
      v[j] = at[j] >= 0 ? load_pair(kp + at[j], far[j]) : make_float2(0.f, 0.f);
      w[j] = a.k_weight && at[j] >= 0 ? make_float2(a.k_weight[at[j]], a.k_weight[at[j] + far[j]]) : make_float2(1.f, 1.f);
      b[j] = a.k_bias && at[j] >= 0 ? make_float2(a.k_bias[at[j]], a.k_bias[at[j] + far[j]]) : make_float2(0.f, 0.f);
    }
    const float d = static_cast<float>(a.d_I), inv_d = 1.f / d;
    if (a.k_norm == LSA_NORM_LAYER) {
      const float mean = mean_of(warp_sum((v[0].x + v[0].y) + (v[1].x + v[1].y) + (v[2].x + v[2].y)), d, inv_d);
      #pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at[j] >= 0) v[j] = make_float2(v[j].x - mean, v[j].y - mean);
    }
    if (a.k_norm != LSA_NORM_NONE) {
      const float s = fmaf(v[0].x, v[0].x, v[0].y * v[0].y) +
                      (fmaf(v[1].x, v[1].x, v[1].y * v[1].y) + fmaf(v[2].x, v[2].x, v[2].y * v[2].y));
      const float q = rsqrtf(warp_sum(s) * inv_d + a.k_eps);
      #pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at[j] >= 0) v[j] = make_float2(fmaf(v[j].x * q, w[j].x, b[j].x), fmaf(v[j].y * q, w[j].y, b[j].y));
    }
    if (turn) {
      const float2 cs = rope_cs(pos, fr, a.mul);
      v[0] = make_float2(v[0].x * cs.x - v[0].y * cs.y, v[0].y * cs.x + v[0].x * cs.y);
    }
    if (FP8) {
      float m = 0.f;
      #pragma unroll
      for (int j = 0; j < 3; ++j) m = max_nan(m, max_nan(fabsf(v[j].x), fabsf(v[j].y)));
      const float2 sc = row_scale(group_max<32>(m));
      if (!write) return;
      uint8_t* o = static_cast<uint8_t*>(a.kc) + slot * a.d_I;
      const float inv = tiny_row(v, sc);
      #pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at[j] >= 0) store_codes(o + at[j], far[j], codes2(v[j], both(inv)));
      if (lane == 0) a.k_scale[slot] = sc.x;
    } else if (write) {
      uint16_t* o = static_cast<uint16_t*>(a.kc) + slot * a.d_I;
      #pragma unroll
      for (int j = 0; j < 3; ++j)
        if (at[j] >= 0) store_pair(o + at[j], far[j], v[j]);
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
  a.off = off;
  a.R = freqs ? R : 0;
  a.half = layout == LSA_ROPE_HALF;
  a.eps = eps;
  a.mul = mul;
  const bool fp8 = dtype == LSA_FP8_E4M3;
  a.only_rotary = !fp8 && norm == LSA_NORM_NONE && x == y && ldt == yldt && ldh == yldh;
  // lanes a row: two 16-byte chunks a lane (a rotary pair of chunks lies in one lane), three where that leaves none idle
  const int n = D >> 3;
  int G = 32, it = n <= 64 ? 2 : n <= 96 && a.R / 16 <= 32 ? 3 : 4;
  for (int g = 16; g >= 2; g /= 2) {
    if (n <= 2 * g) {
      G = g;
      it = 2;
    } else if (n == 3 * g && g >= 4 && a.R / 16 <= g) {
      G = g;
      it = 3;
      break;
    }
  }
  // a block's row slots go to one token as far as it has heads; where the blocks are many, a block takes more of a
  // token's heads, then more tokens, up to two table entries a thread
  const int slots = NR_THREADS / G, many = 4 * sm_count();
  a.spt_log = 0;
  while ((1 << a.spt_log) < slots && (1 << a.spt_log) < H) ++a.spt_log;
  const int spt = 1 << a.spt_log, NT = slots >> a.spt_log;
  a.HB = spt;
  a.TB = 1;
  while (a.HB < H && a.HB < 4 * spt && cdiv(T, NT) * cdiv(H, 2 * a.HB) >= many) a.HB *= 2;
  while (a.HB * a.TB < 8 * spt && NT * a.TB * a.R <= 1024 && cdiv(T, 2 * a.TB * NT) * cdiv(H, a.HB) >= many) a.TB *= 2;
  const int64_t gx = cdiv(T, NT * a.TB);
  if (gx > 0x7FFFFFFF) return LSA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(NT) * a.TB * (a.R / 2) * sizeof(float2) + (norm == LSA_NORM_NONE ? 0 : 8 * D);
  const dim3 g(static_cast<unsigned>(gx), static_cast<unsigned>(cdiv(H, a.HB)));
  cudaError_t e = cudaErrorInvalidValue;
  if (it == 2) {
    if (G == 2) e = go_norm_rope<2, 2>(a, norm, fp8, g, smem, s);
    else if (G == 4) e = go_norm_rope<4, 2>(a, norm, fp8, g, smem, s);
    else if (G == 8) e = go_norm_rope<8, 2>(a, norm, fp8, g, smem, s);
    else if (G == 16) e = go_norm_rope<16, 2>(a, norm, fp8, g, smem, s);
    else e = go_norm_rope<32, 2>(a, norm, fp8, g, smem, s);
  } else if (it == 3) {
    if (G == 4) e = go_norm_rope<4, 3>(a, norm, fp8, g, smem, s);
    else if (G == 8) e = go_norm_rope<8, 3>(a, norm, fp8, g, smem, s);
    else if (G == 16) e = go_norm_rope<16, 3>(a, norm, fp8, g, smem, s);
    else e = go_norm_rope<32, 3>(a, norm, fp8, g, smem, s);
  } else {
    e = go_norm_rope<32, 4>(a, norm, fp8, g, smem, s);
  }
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
