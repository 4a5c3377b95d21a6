// qsa_rope.cu -- norms of the new queries and keys with their rotation,
// declared in include/qsa_rope.h.
//
// A head of D elements lies in the lanes of half a warp (D = 128) or of what
// D/8 rounds up to, 16 bytes a lane: the sum of squares is a few shuffles, and a
// pair whose elements lie rot_dim/2 apart is one more.  A warp takes heads of one
// token, since their angles are the same: its lanes form the sines and cosines once,
// each its share, and turn every head with them.
//
// Angles.  A turn is 2^64: a frequency f becomes F = f / (2 pi) * 2^64 (its 24
// bits times 1/(2 pi) to 64 bits, an integer product), and position * F modulo
// 2^64 is the angle modulo one turn, without any rounding that grows with the
// position (binary32 products are off by a radian at position 2^24).  Binary64
// would do as well; its rate here is a sixtieth of the integer one.
//
// Bytes bound it: each element is read and written once.  16344 tokens of 40 heads
// of 128: pairs side by side 56.5 us (5.9 TB/s), half a head apart 70 (4.8 TB/s: two
// shuffles more a pair, and the 80 registers of three CTAs an SM leave 96 to 112 bytes
// a thread on the stack, where the other order has 8 at most); each lane forming all
// angles of its own elements, with heads of q and k in one loop, 78 and 106; two and
// four CTAs an SM 65 and 70, 71 and 98.
#include "qsa_cache_host.h"
#include "qsa_device.cuh"
#include "qsa_host.h"
#include "qsa_internal.h"
#include "qsa_rope.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace qsa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 3;       // of an SM
constexpr int kRopeUnroll = 4;     // heads of a lane in flight

struct RopeParams {
  const unsigned char* in[2];      // q, k
  unsigned char* out[2];
  int64_t in_tok[2], in_head[2], out_tok[2], out_head[2];   // bytes
  const void* weight[2];
  int32_t heads[2];
  int32_t dim, rot;
  float inv_dim, eps;
  const int64_t* positions;
  const float* inv_freq;
  int64_t tokens;
  int32_t split;                   // warps that share a token
};

// f / (2 pi) modulo 1, times 2^64.
__device__ __forceinline__ uint64_t turns(float f) {
  constexpr uint64_t kInvTwoPi = 0x28be60db9391054aull;     // 2^64 / (2 pi)
  const uint32_t u = __float_as_uint(f), e = (u >> 23) & 255u;
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  const int shift = 150 - (int)max(e, 1u);                  // f = m * 2^-shift
  uint64_t t;
  if (shift <= 0) t = shift > -64 ? lo << -shift : 0;
  else if (shift < 64) t = lo >> shift | hi << (64 - shift);
  else t = shift < 128 ? hi >> (shift - 64) : 0;
  return u >> 31 ? 0 - t : t;
}

__device__ __forceinline__ float2 fmul2(float2 a, float2 b) { return ffma2(a, b, make_float2(-0.f, -0.f)); }

template <typename T>
__device__ __forceinline__ float2 widen(uint32_t x) {
  if constexpr (__is_same(T, __nv_bfloat16))
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  else
    return h2f2(x);
}
template <typename T>
__device__ __forceinline__ uint32_t narrow(float lo, float hi) {
  uint32_t r;
  if constexpr (__is_same(T, __nv_bfloat16))
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// L lanes a head, 8 elements a lane.
template <typename T, typename WT, int L, bool kPairs>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeParams p) {
  constexpr int kHeads = 32 / L;                            // heads of a warp at a time
  __shared__ uint64_t s_freq[QSA_ROPE_MAX_DIM / 2];
  __shared__ __align__(16) float2 s_angles[kRopeThreads / 32][QSA_ROPE_MAX_DIM / 2];
  float2* angles = s_angles[threadIdx.x >> 5];              // cosine and sine
  const int lane = threadIdx.x & 31, piece = lane % L;
  const int64_t warps = (int64_t)gridDim.x * (kRopeThreads / 32);
  const int64_t warp = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int half = p.rot / 16;                              // pieces of half the turned elements
  const bool there = piece * 8 < p.dim, turned = piece * 8 < p.rot;
  const bool upper = piece >= half;
  // the lane that holds the other elements of this lane's pairs
  const int other = kPairs || !turned ? lane : upper ? lane - half : lane + half;
  float2 w[2][4];
  pdl_wait();          // whatever is read may be the kernel's before it
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) s_freq[i] = turns(p.inv_freq[i]);
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const WT* v = static_cast<const WT*>(p.weight[x]) + piece * 8 + i * 2;
      w[x][i] = there && p.weight[x] ? make_float2((float)v[0], (float)v[1]) : make_float2(1.f, 1.f);
    }
  const int64_t items = p.tokens * p.split;
  for (int64_t item = warp; item < items; item += warps) {
    const int64_t t = item / p.split;
    const int part = (int)(item - t * p.split);
    const int64_t pos = p.positions[t];
    if (pos < 0) continue;
    __syncwarp();                                           // the last token's have been read
#pragma unroll 2
    for (int i = lane; i < p.rot / 2; i += 32) {
      // half turns in [-1, 1)
      const float x = (float)(int32_t)(uint32_t)((uint64_t)pos * s_freq[i] >> 32) * 0x1p-31f;
      float2 a;
      sincospif(x, &a.y, &a.x);
      angles[i] = a;
    }
    __syncwarp();
    // a rotated element: its own times the cosine, the pair's other one times the sine
    // (neighbours, or the same element of another lane); cosines and sines as pairs of
    // neighbouring elements
    float2 c[4], s[4];
    const float4* mine = reinterpret_cast<const float4*>(
        angles + (!turned ? 0 : kPairs ? piece * 4 : (upper ? piece - half : piece) * 8));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kPairs) {
        const float4 a = mine[i / 2];
        const float2 b = i & 1 ? make_float2(a.z, a.w) : make_float2(a.x, a.y);
        c[i] = make_float2(b.x, b.x);
        s[i] = make_float2(-b.y, b.y);
      } else {
        const float4 a = mine[i];
        c[i] = make_float2(a.x, a.z);
        s[i] = upper ? make_float2(a.y, a.w) : make_float2(-a.y, -a.w);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int heads = p.heads[x], step = p.split * kHeads;
      const int64_t in_step = step * p.in_head[x], out_step = step * p.out_head[x];
      int h = part * kHeads + lane / L;
      const unsigned char* in = p.in[x] + t * p.in_tok[x] + h * p.in_head[x] + piece * 16;
      unsigned char* out = p.out[x] + t * p.out_tok[x] + h * p.out_head[x] + piece * 16;
      for (int h0 = part * kHeads; h0 < heads; h0 += step * kRopeUnroll) {
        uint4 v[kRopeUnroll];
#pragma unroll
        for (int k = 0; k < kRopeUnroll; ++k) {
          v[k] = make_uint4(0, 0, 0, 0);
          if (there && h + k * step < heads) v[k] = *reinterpret_cast<const uint4*>(in + k * in_step);
        }
#pragma unroll
        for (int k = 0; k < kRopeUnroll; ++k) {
          if (h0 + k * step >= heads) break;                // the whole warp's
          const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          float2 y[4], sum2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = widen<T>(u[i]);
            sum2 = ffma2(y[i], y[i], sum2);
          }
          float sum = sum2.x + sum2.y;
#pragma unroll
          for (int i = 1; i < L; i <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
          const float r = rsqrtf(fmaf(sum, p.inv_dim, p.eps));
          uint32_t z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = fmul2(y[i], fmul2(w[x][i], make_float2(r, r)));
            float2 o;
            if constexpr (kPairs) o = make_float2(y[i].y, y[i].x);
            else o = make_float2(__shfl_sync(0xffffffffu, y[i].x, other),
                                 __shfl_sync(0xffffffffu, y[i].y, other));
            const float2 q = ffma2(o, s[i], fmul2(y[i], c[i]));
            z[i] = turned ? narrow<T>(q.x, q.y) : narrow<T>(y[i].x, y[i].y);
          }
          if (there && h + k * step < heads)
            *reinterpret_cast<uint4*>(out + k * out_step) = make_uint4(z[0], z[1], z[2], z[3]);
        }
        h += step * kRopeUnroll;
        in += in_step * kRopeUnroll;
        out += out_step * kRopeUnroll;
      }
    }
  }
}

template <typename T, typename WT, int L>
cudaError_t launch_rope_lanes(const RopeParams& p, bool pairs, int grid, cudaStream_t st) {
  return pairs ? launch_after(rope_kernel<T, WT, L, true>, dim3(grid), dim3(kRopeThreads), 0, st, p)
               : launch_after(rope_kernel<T, WT, L, false>, dim3(grid), dim3(kRopeThreads), 0, st, p);
}

template <typename T, typename WT>
cudaError_t launch_rope(const RopeParams& p, int lanes, bool pairs, int grid, cudaStream_t st) {
  switch (lanes) {
    case 1: return launch_rope_lanes<T, WT, 1>(p, pairs, grid, st);
    case 2: return launch_rope_lanes<T, WT, 2>(p, pairs, grid, st);
    case 4: return launch_rope_lanes<T, WT, 4>(p, pairs, grid, st);
    case 8: return launch_rope_lanes<T, WT, 8>(p, pairs, grid, st);
    case 16: return launch_rope_lanes<T, WT, 16>(p, pairs, grid, st);
    default: return launch_rope_lanes<T, WT, 32>(p, pairs, grid, st);
  }
}

// A [tokens, heads, dim] view: bytes of a token from its first to its last
// element, and between tokens.
struct View {
  cache_host::Span all;
  int64_t inner, step, tokens;
};

// Whether two views share no byte: apart, or rows of one width side by side.
bool apart(const View& a, const View& b) {
  if (!cache_host::overlaps(a.all, b.all)) return true;
  if (a.tokens <= 1 || b.tokens <= 1 || a.step != b.step) return false;
  const int64_t d = (int64_t)((b.all.lo - a.all.lo) % (uintptr_t)a.step);
  const int64_t off =
      b.all.lo >= a.all.lo ? d : a.step - (int64_t)((a.all.lo - b.all.lo) % (uintptr_t)a.step);
  const int64_t o = off == a.step ? 0 : off;
  return o >= a.inner && o + b.inner <= a.step;
}

}  // namespace
}  // namespace qsa

extern "C" qsa_status qsa_qk_norm_rope(
    const void* q, const void* k, qsa_dtype dtype, int64_t num_tokens, int64_t q_heads,
    int64_t k_heads, int64_t head_dim, const int64_t q_strides[3], const int64_t k_strides[3],
    const void* q_weight, const void* k_weight, qsa_dtype weight_dtype, float eps,
    const int64_t* positions, const float* inv_freq, int64_t rot_dim, int interleaved, void* q_out,
    void* k_out, const int64_t q_out_strides[3], const int64_t k_out_strides[3],
    qsa_stream_t stream) {
  using namespace qsa;
  using namespace qsa::cache_host;
  if (dtype != QSA_DT_F16 && dtype != QSA_DT_BF16) return QSA_ERR_DTYPE;
  const bool weights = q_weight || k_weight;
  if (weights && weight_dtype != QSA_DT_F32 && weight_dtype != dtype) return QSA_ERR_DTYPE;
  if (head_dim < 8 || head_dim > QSA_ROPE_MAX_DIM || head_dim % 8 != 0) return QSA_ERR_SHAPE;
  if (num_tokens < 0 || num_tokens > INT32_MAX || q_heads < 0 || q_heads > QSA_ROPE_MAX_HEADS ||
      k_heads < 0 || k_heads > QSA_ROPE_MAX_HEADS)
    return QSA_ERR_SHAPE;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0) return QSA_ERR_SHAPE;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return QSA_ERR_CONTRACT;
  RopeParams p{};
  View in[2], out[2];
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const int64_t* ss[2] = {q_strides, k_strides};
  const int64_t* ds[2] = {q_out_strides, k_out_strides};
  const int64_t heads[2] = {q_heads, k_heads};
  for (int x = 0; x < 2; ++x) {
    p.heads[x] = (int32_t)heads[x];
    if (heads[x] == 0 || num_tokens == 0) {
      in[x] = out[x] = View{Span{0, 0}, 0, 0, 0};
      continue;
    }
    if (!ss[x] || !ds[x]) return QSA_ERR_NULL;
    const int64_t shape[3] = {num_tokens, heads[x], head_dim};
    if (!strides_ok(shape, ss[x], 3, 2) || !strides_ok(shape, ds[x], 3, 2) ||
        !separate(shape, ds[x], 3))
      return QSA_ERR_STRIDE;
    const int64_t ix = extent(shape, ss[x], 3, 2), ox = extent(shape, ds[x], 3, 2);
    if (ix < 0 || ox < 0) return QSA_ERR_STRIDE;
    if (!src[x] || !dst[x]) return QSA_ERR_NULL;
    if (!aligned(src[x], 16) || !aligned(dst[x], 16)) return QSA_ERR_ALIGN;
    const auto step = [&](const int64_t* s, int i) { return shape[i] > 1 ? s[i] * 2 : 0; };
    p.in_tok[x] = step(ss[x], 0);
    p.in_head[x] = step(ss[x], 1);
    p.out_tok[x] = step(ds[x], 0);
    p.out_head[x] = step(ds[x], 1);
    in[x] = View{span(src[x], ix), (heads[x] - 1) * p.in_head[x] + head_dim * 2, p.in_tok[x], num_tokens};
    out[x] = View{span(dst[x], ox), (heads[x] - 1) * p.out_head[x] + head_dim * 2, p.out_tok[x],
                  num_tokens};
    p.in[x] = static_cast<const unsigned char*>(src[x]);
    p.out[x] = static_cast<unsigned char*>(dst[x]);
  }
  if (num_tokens == 0 || q_heads + k_heads == 0) return QSA_OK;
  if (!positions || (rot_dim > 0 && !inv_freq)) return QSA_ERR_NULL;
  const uintptr_t wa = weight_dtype == QSA_DT_F32 ? 4 : 2;
  if (!aligned(positions, 8) || !aligned(inv_freq, 4) ||
      (weights && (!aligned(q_weight, wa) || !aligned(k_weight, wa))))
    return QSA_ERR_ALIGN;
  const Span small[4] = {span(q_weight, head_dim * (int64_t)wa), span(k_weight, head_dim * (int64_t)wa),
                         span(positions, num_tokens * 8), span(inv_freq, rot_dim / 2 * 4)};
  for (int x = 0; x < 2; ++x) {
    if (out[x].tokens == 0) continue;
    const bool in_place = src[x] == dst[x] && p.in_tok[x] == p.out_tok[x] && p.in_head[x] == p.out_head[x];
    if (!in_place && in[x].tokens && !apart(out[x], in[x])) return QSA_ERR_ALIAS;
    if (in[1 - x].tokens && !apart(out[x], in[1 - x])) return QSA_ERR_ALIAS;
    for (const Span& s : small)
      if (overlaps(out[x].all, s)) return QSA_ERR_ALIAS;
  }
  if (out[0].tokens && out[1].tokens && !apart(out[0], out[1])) return QSA_ERR_ALIAS;
  p.weight[0] = q_weight;
  p.weight[1] = k_weight;
  p.dim = (int32_t)head_dim;
  p.rot = (int32_t)rot_dim;
  p.inv_dim = 1.f / (float)head_dim;
  p.eps = eps;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.tokens = num_tokens;
  int lanes = 1;
  while (lanes * 8 < head_dim) lanes *= 2;
  bind_calling_thread();
  // a token's heads over several warps where there are few tokens, each of which forms
  // the angles again (256 tokens of 40 heads of 128: 5.0 us with up to 8 warps an SM,
  // 6.5 with 4, 5.3 with 16, 7.4 with 32)
  const int64_t rounds = (q_heads + k_heads + 32 / lanes - 1) / (32 / lanes);
  constexpr int64_t kWarps = 152 * 8;
  p.split = (int32_t)std::max<int64_t>(1, std::min<int64_t>(rounds, kWarps / num_tokens));
  const int64_t ctas = (num_tokens * p.split + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int grid = (int)std::min<int64_t>(ctas, 152 * kRopeCtas);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool pairs = interleaved != 0, wide = weight_dtype == QSA_DT_F32;
  cudaError_t e;
  if (dtype == QSA_DT_BF16)
    e = wide ? launch_rope<__nv_bfloat16, float>(p, lanes, pairs, grid, st)
             : launch_rope<__nv_bfloat16, __nv_bfloat16>(p, lanes, pairs, grid, st);
  else
    e = wide ? launch_rope<__half, float>(p, lanes, pairs, grid, st)
             : launch_rope<__half, __half>(p, lanes, pairs, grid, st);
  return e == cudaSuccess ? QSA_OK : QSA_ERR_CUDA;
}
