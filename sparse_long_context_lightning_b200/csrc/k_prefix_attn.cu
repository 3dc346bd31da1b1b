// Dense absorbed-MQA attention of a batch behind one shared prefix, each query with its own tokens in pages.
//
//   o = sum_k e^{scale q.k - m} v_k / l,  l = sum_k e^{scale q.k - m},  lse = m + ln l,  v = the first 512 dims of k,
// over the Lp rows of the prefix (the same for every query) and own_len[b] rows behind them (block table).
//
// One block a query and eight of its heads, a warp a head: tiles of 32 keys in shared memory serve the eight heads,
// a lane forms one key's logit, and a lane holds 16 of the 512 output dims.  CUDA cores, so 2 (576 + 512) flops a
// (head, key) bound it, and every block reads the whole prefix.
#include "lsa_common.cuh"
#include "sm100.cuh"

namespace lsa {
namespace {

__device__ int g_prefix_check;  // set when own_len was outside [0, the table's columns * page] or a page id was bad

constexpr int PA_THREADS = 256;
constexpr int PA_T = 32;        // keys of a tile
constexpr int PA_LD = 576 + 8;  // bf16 elements of a tile's row: 16-byte reads of 8 rows meet every bank once
constexpr int PA_SMEM = 8 * 576 * 4 + PA_T * PA_LD * 2;

struct PaArgs {
  const uint16_t* q;
  const uint16_t* prefix;
  const uint16_t* pages;
  const int32_t* own_len;  // [B], or NULL: no own tokens
  const int32_t* table;    // [B, table_ld] page ids
  int64_t table_ld;
  int page_shift;
  int64_t n_pages;
  int64_t cap;  // most own tokens
  int64_t Lp;
  int H;
  float scale;
};

__global__ void __launch_bounds__(PA_THREADS) k_prefix_attn(const PaArgs a, uint16_t* __restrict__ out,
                                                            float* __restrict__ lse) {
  extern __shared__ __align__(16) unsigned char smem[];
  float* q_s = reinterpret_cast<float*>(smem);
  uint16_t* k_s = reinterpret_cast<uint16_t*>(smem + 8 * 576 * 4);
  sm100::pdl_wait();
  sm100::pdl_launch_dependents();
  const int groups = (a.H + 7) / 8;
  const int64_t b = blockIdx.x / groups;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = static_cast<int>(blockIdx.x % groups) * 8, h = h0 + warp;
  for (int i = threadIdx.x; i < 8 * 576; i += PA_THREADS)
    q_s[i] = h0 + i / 576 < a.H ? bf16_bits_to_f32(a.q[(b * a.H + h0) * 576 + i]) : 0.f;
  int64_t own = a.own_len ? a.own_len[b] : 0;
  if (own < 0 || own > a.cap) {
    if (threadIdx.x == 0) atomicExch(&g_prefix_check, 1);
    own = own < 0 ? 0 : a.cap;
  }
  const int64_t n = a.Lp + own;
  float m = -INFINITY, l = 0.f, o[16];
  #pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  for (int64_t k0 = 0; k0 < n; k0 += PA_T) {
    __syncthreads();
    for (int i = threadIdx.x; i < PA_T * 72; i += PA_THREADS) {
      const int64_t key = k0 + i / 72;
      const uint16_t* row = nullptr;
      if (key < a.Lp) {
        row = a.prefix + key * 576;
      } else if (key < n) {
        const int64_t t = key - a.Lp;
        const int32_t pg = a.table[b * a.table_ld + (t >> a.page_shift)];
        if (pg >= 0 && pg < a.n_pages)
          row = a.pages + ((static_cast<int64_t>(pg) << a.page_shift) + (t & ((1 << a.page_shift) - 1))) * 576;
        else
          atomicExch(&g_prefix_check, 1);
      }
      *reinterpret_cast<uint4*>(k_s + (i / 72) * PA_LD + (i % 72) * 8) =
          row ? reinterpret_cast<const uint4*>(row)[i % 72] : make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    float z = 0.f;
    for (int c = 0; c < 72; ++c) {
      const uint4 v = *reinterpret_cast<const uint4*>(k_s + lane * PA_LD + c * 8);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        z = fmaf(q_s[warp * 576 + c * 8 + 2 * i], __uint_as_float(u[i] << 16), z);
        z = fmaf(q_s[warp * 576 + c * 8 + 2 * i + 1], __uint_as_float(u[i] & 0xFFFF0000u), z);
      }
    }
    z = k0 + lane < n ? z * a.scale : -INFINITY;
    const float mn = fmaxf(m, warp_max(z));
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = expf(m - ref), p = expf(z - ref);
    l = l * alpha + warp_sum(p);
    m = mn;
    #pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= alpha;
    const int keys = static_cast<int>(n - k0 < PA_T ? n - k0 : PA_T);
    for (int k = 0; k < keys; ++k) {
      const float pk = __shfl_sync(0xffffffffu, p, k);
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(k_s + k * PA_LD + 64 * i + 2 * lane);
        o[2 * i] = fmaf(pk, __uint_as_float(v << 16), o[2 * i]);
        o[2 * i + 1] = fmaf(pk, __uint_as_float(v & 0xFFFF0000u), o[2 * i + 1]);
      }
    }
  }
  if (h >= a.H) return;
  const float inv = l != 0.f ? 1.f / l : 0.f;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(o[2 * i] * inv, o[2 * i + 1] * inv);
    *reinterpret_cast<uint32_t*>(out + (b * a.H + h) * 512 + 64 * i + 2 * lane) = *reinterpret_cast<const uint32_t*>(&p);
  }
  if (lse && lane == 0) lse[b * a.H + h] = l != 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t prefix_attn_ws_bytes(int64_t B, int H) { return B > 0 && H > 0 ? 256 : 0; }

int launch_prefix_attn(const void* q, int64_t B, int H, const void* prefix, int64_t Lp, const void* pages,
                       int64_t n_pages, int page, const int32_t* table, int64_t table_ld, const int32_t* own_len,
                       float scale, void* out, float* lse, void* ws, cudaStream_t s) {
  (void)ws;
  PaArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.prefix = static_cast<const uint16_t*>(prefix);
  a.pages = static_cast<const uint16_t*>(pages);
  a.own_len = own_len;
  a.table = table;
  a.table_ld = table_ld;
  a.page_shift = 0;
  while ((1 << a.page_shift) < page) ++a.page_shift;
  a.n_pages = n_pages;
  a.cap = table_ld * page;
  a.Lp = Lp;
  a.H = H;
  a.scale = scale;
  LSA_CUDA_TRY(func_smem_once(reinterpret_cast<const void*>(k_prefix_attn), PA_SMEM));
  return cuda_status(launch_pdl(k_prefix_attn, dim3(static_cast<unsigned>(B * ((H + 7) / 8))), dim3(PA_THREADS), PA_SMEM,
                                s, 0u, a, static_cast<uint16_t*>(out), lse));
}

// The kernel's flags, read and cleared: give-up (it has no waits) and device check; -1: CUDA error.
int take_prefix_flags(int* check) {
  int c = 0;
  if (cudaMemcpyFromSymbol(&c, g_prefix_check, sizeof(int)) != cudaSuccess) return -1;
  const int zero = 0;
  if (c != 0 && cudaMemcpyToSymbol(g_prefix_check, &zero, sizeof(int)) != cudaSuccess) return -1;
  *check = c;
  return 0;
}

}  // namespace lsa
