// Rotary positions: the pairs of dims of every query and key head turned by
// t * freq[i] (the rotation that the attention calls expect to have been
// applied; EAGLE-2 article, position encoding of the flattened tree).
//
// Bound by memory: each value is read once and written once, in 16-byte
// accesses (8192 rows of 72 heads of 128, bf16: 49.7 us = 6.07 TB/s).  A block takes a token; it finds the sines and cosines once, for
// all heads, while its first values are on their way.
// The angle in turns is t * (freq / 2 pi) modulo 1: freq / 2 pi, an fp64 product
// (off by freq 2^-55 of a turn, the constant's rounding included), is cut to a
// multiple of 2^-64, and that times t in 64-bit integers is exact and wraps by
// itself.  So an angle is off by t times that product's error and nothing
// else (2^-24 of a turn at position 2^31 for freq = 1), and no fp64 arithmetic
// is left per token and dim but the one product that makes the integer.
#include <cuda_bf16.h>

#include "et_common.cuh"

namespace et {
namespace {

constexpr int kRoMaxDim = 512;

struct RotaryArgs {
  int rows, Hq, H, d, rot, layout;          // H = Hq + Hkv
  int units;                                // units per head (see below)
  float factor;
  long long qs, ks, qos, kos;
  const int32_t *positions;
  const double *freq;
  const void *q, *k;
  void *qo, *ko;
};

template <typename T>
struct Vec {};  // 16 bytes
template <>
struct Vec<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void get(const uint4 &v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void get(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A unit is two vectors of a head: vector u and the one that holds the dims
// rot / 2 further (half layout), or vectors 2 u and 2 u + 1 (pairs, and the
// dims behind rot, which are copied).
template <typename T, bool HALF, int NT>
__global__ void __launch_bounds__(NT, 2048 / NT) k_rotary(const RotaryArgs a) {
  constexpr int N = Vec<T>::n;
  __shared__ float2 s_turn[kRoMaxDim / 2];  // factor * (cos, sin)
  pdl_wait();
  pdl_trigger();
  const int half = a.rot >> 1, row = blockIdx.x, pos = a.positions[row];
  if (pos < 0) return;  // no token
  const int rot_units = HALF ? half / N : a.rot / (2 * N), per = a.H * a.units;
  struct Unit {
    const T *in;
    T *out;
    int o0, o1;  // its vectors
    bool turn;
  };
  auto unit = [&](int y) -> Unit {
    const int h = y / a.units, u = y - h * a.units;
    const bool is_q = h < a.Hq;
    Unit x;
    x.in = is_q ? static_cast<const T *>(a.q) + row * a.qs + (long long)h * a.d
                : static_cast<const T *>(a.k) + row * a.ks + (long long)(h - a.Hq) * a.d;
    x.out = is_q ? static_cast<T *>(a.qo) + row * a.qos + (long long)h * a.d
                 : static_cast<T *>(a.ko) + row * a.kos + (long long)(h - a.Hq) * a.d;
    x.turn = u < rot_units;
    if (HALF && x.turn) {
      x.o0 = u * N;
      x.o1 = x.o0 + half;
    } else {
      x.o0 = (HALF ? a.rot : 0) + 2 * N * (HALF ? u - rot_units : u);
      x.o1 = x.o0 + N;
    }
    return x;
  };
  auto load = [&](const Unit &x, uint4 &v0, uint4 &v1) {
    v0 = *reinterpret_cast<const uint4 *>(x.in + x.o0);
    v1 = x.o1 < a.d ? *reinterpret_cast<const uint4 *>(x.in + x.o1) : make_uint4(0u, 0u, 0u, 0u);
  };
  // the first unit's values are on their way while the sines are found
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  if (threadIdx.x < per) load(unit(threadIdx.x), v0, v1);
  for (int i = threadIdx.x; i < half; i += NT) {
    double turns = a.freq[i] * 0.15915494309189533577;  // 1 / 2 pi
    turns -= floor(turns);
    const unsigned long long step = (unsigned long long)(turns * 18446744073709551616.0);  // 2^64; 1.0 saturates
    const long long at = (long long)(step * (unsigned long long)(long long)pos);  // turns modulo 1, in [-1/2, 1/2)
    float s, c;
    sincospif((float)at * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    s_turn[i] = make_float2(c * a.factor, s * a.factor);
  }
  __syncthreads();
  for (int y = threadIdx.x; y < per; y += NT) {
    const Unit x = unit(y);
    if (y != threadIdx.x) load(x, v0, v1);
    uint4 w0 = v0, w1 = v1;
    if (x.turn) {
      float p[N], r[N];
      Vec<T>::get(v0, p);
      Vec<T>::get(v1, r);
      if (HALF) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 f = s_turn[x.o0 + e];
          const float a0 = p[e], b0 = r[e];
          p[e] = a0 * f.x - b0 * f.y;
          r[e] = b0 * f.x + a0 * f.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          const float2 f = s_turn[(x.o0 + e) >> 1], g = s_turn[(x.o1 + e) >> 1];
          const float a0 = p[e], b0 = p[e + 1], a1 = r[e], b1 = r[e + 1];
          p[e] = a0 * f.x - b0 * f.y;
          p[e + 1] = b0 * f.x + a0 * f.y;
          r[e] = a1 * g.x - b1 * g.y;
          r[e + 1] = b1 * g.x + a1 * g.y;
        }
      }
      w0 = Vec<T>::put(p);
      w1 = Vec<T>::put(r);
    }
    *reinterpret_cast<uint4 *>(x.out + x.o0) = w0;
    if (x.o1 < a.d) *reinterpret_cast<uint4 *>(x.out + x.o1) = w1;
  }
}

template <typename T>
et_status launch_rotary(RotaryArgs a, cudaStream_t st) {
  constexpr int N = Vec<T>::n;
  const bool half = a.layout == ET_ROTARY_HALF;
  // vectors behind rot go two to a unit, the last one alone if they are odd in number
  a.units = half ? a.rot / (2 * N) + (a.d - a.rot + 2 * N - 1) / (2 * N) : (a.d + 2 * N - 1) / (2 * N);
  // Many rows: blocks of four warps, as many as an SM holds, keep more loads in flight (8192 rows of 72 heads, bf16: 49.7 us
  // in blocks of 128, 53.2 of 256, 62.9 of 512).  Less than a wave of those: a row's units spread over more threads (61 rows
  // of 64 heads: 3.0 us in blocks of 512, 3.9 of 128; 1503 rows of 80 heads in fp32: 12.0 and 13.4)
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) sms = 152;
  cudaGetLastError();
  const dim3 grid(a.rows);
  if (a.rows >= 16 * sms)
    return half ? et_launch(k_rotary<T, true, 128>, grid, dim3(128), 0, st, 0, a)
                : et_launch(k_rotary<T, false, 128>, grid, dim3(128), 0, st, 0, a);
  return half ? et_launch(k_rotary<T, true, 512>, grid, dim3(512), 0, st, 0, a)
              : et_launch(k_rotary<T, false, 512>, grid, dim3(512), 0, st, 0, a);
}

bool stride_ok(long long stride, int H, const et_rotary_shape *s) {
  const int es = s->dtype == ET_BF16 ? 2 : 4;
  return stride >= (long long)H * s->d && stride < (1ll << 40) && stride * es % 16 == 0;
}

}  // namespace
}  // namespace et

using namespace et;

extern "C" et_status et_rotary(const et_rotary_shape *s, const int32_t *positions, const double *freq, const void *q,
                               const void *k, void *q_out, void *k_out, et_stream_t stream) {
  ET_RETURN_IF(!s || !positions || !freq || !q || !q_out || (k == nullptr) != (k_out == nullptr), ET_ERR_INVALID_ARG);
  ET_RETURN_IF(s->rows < 1 || s->Hq < 1 || s->Hkv < 0 || (s->Hkv > 0) != (k != nullptr) || s->d < 8 || s->d % 8 ||
                   s->rot < 16 || s->rot % 16 || s->rot > s->d || !(fabsf(s->factor) <= FLT_MAX) ||
                   (s->layout != ET_ROTARY_HALF && s->layout != ET_ROTARY_PAIRS) ||
                   (s->dtype != ET_BF16 && s->dtype != ET_F32),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(s->d > kRoMaxDim || s->Hq > 65535 || s->Hkv > 65535, ET_ERR_UNSUPPORTED);
  ET_RETURN_IF(!stride_ok(s->q_stride, s->Hq, s) || !stride_ok(s->q_out_stride, s->Hq, s) ||
                   (k && (!stride_ok(s->k_stride, s->Hkv, s) || !stride_ok(s->k_out_stride, s->Hkv, s))),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(!et_aligned(q, 16) || !et_aligned(q_out, 16) || !et_aligned(k, 16) || !et_aligned(k_out, 16) ||
                   !et_aligned(positions, 4) || !et_aligned(freq, 8),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF((q == q_out && s->q_stride != s->q_out_stride) || (k && k == k_out && s->k_stride != s->k_out_stride),
               ET_ERR_INVALID_ARG);
  RotaryArgs a = {};
  a.rows = s->rows; a.Hq = s->Hq; a.H = s->Hq + s->Hkv; a.d = s->d; a.rot = s->rot; a.layout = s->layout;
  a.factor = s->factor;
  a.qs = s->q_stride; a.ks = s->k_stride; a.qos = s->q_out_stride; a.kos = s->k_out_stride;
  a.positions = positions; a.freq = freq; a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
  return s->dtype == ET_BF16 ? launch_rotary<__nv_bfloat16>(a, (cudaStream_t)stream)
                             : launch_rotary<float>(a, (cudaStream_t)stream);
}

extern "C" et_status et_rotary_frequencies(const et_rope_cfg *c, double *freq, float *factor) {
  ET_RETURN_IF(!c || !freq || !factor || c->rot < 2 || c->rot % 2 || c->rot > 512 || !(c->theta > 1.0) ||
                   !(c->theta <= 1e30) || c->scaling < ET_ROPE_PLAIN || c->scaling > ET_ROPE_BANDS,
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(c->scaling != ET_ROPE_PLAIN && !(c->scale >= 1.0 && c->scale <= 1e30), ET_ERR_INVALID_ARG);
  ET_RETURN_IF(c->scaling >= ET_ROPE_RAMP && !(c->trained >= 1.0 && c->trained <= 1e30 && c->slow > 0.0 &&
                                               c->fast > c->slow && c->fast <= 1e30),
               ET_ERR_INVALID_ARG);
  ET_RETURN_IF(c->scaling == ET_ROPE_BASE && c->rot < 4, ET_ERR_INVALID_ARG);
  const double two_pi = 6.283185307179586476925;
  const int n = c->rot / 2;
  const double theta = c->scaling == ET_ROPE_BASE ? c->theta * pow(c->scale, (double)c->rot / (c->rot - 2)) : c->theta;
  *factor = c->scaling == ET_ROPE_RAMP ? (float)(0.1 * log(c->scale) + 1.0) : 1.f;
  // RAMP: the pairs that turn `fast` and `slow` times over `trained` tokens, rounded outward.  The slow end may lie past the last
  // pair, n - 1, when every pair turns more often than `slow` times: the last one keeps its part then
  double lo = 0, hi = 0;
  if (c->scaling == ET_ROPE_RAMP) {
    lo = fmax(0.0, floor(n * log(c->trained / (c->fast * two_pi)) / log(theta)));
    hi = fmin(c->rot - 1.0, ceil(n * log(c->trained / (c->slow * two_pi)) / log(theta)));
  }
  for (int i = 0; i < n; ++i) {
    const double f = pow(theta, -(double)i / n);
    double keep = 1.0;  // share of the unscaled frequency
    if (c->scaling == ET_ROPE_LINEAR) keep = 0.0;
    if (c->scaling == ET_ROPE_RAMP) keep = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
    if (c->scaling == ET_ROPE_BANDS)
      keep = fmin(fmax((c->trained * f / two_pi - c->slow) / (c->fast - c->slow), 0.0), 1.0);
    freq[i] = c->scaling == ET_ROPE_PLAIN || c->scaling == ET_ROPE_BASE ? f : f * keep + f / c->scale * (1.0 - keep);
  }
  return ET_OK;
}
