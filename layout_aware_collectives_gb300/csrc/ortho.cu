// Newton-Schulz orthogonalisation: norms, the first X, and the steps.
#include <cmath>

#include "ortho.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 16;  // elements of a thread and turn of the norm
constexpr int kMaxParts = 64;

struct Sources {
  const void* p[kOrthoTable];
};

template <class T>
__device__ __forceinline__ float element(const T* p);
template <>
__device__ __forceinline__ float element(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float element(const uint16_t* p) {
  return bf16_value(*p);
}

// The whole CTA's; every thread gets it.
template <bool MAX>
__device__ __forceinline__ float reduce(float v, float* shared) {
#pragma unroll
  for (int d = 16; d; d >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, d);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v = MAX ? fmaxf(v, shared[w]) : v + shared[w];
  __syncthreads();
  return v;
}

// A part of a matrix's sum of squares.  Each turn's elements are brought near
// 1 by a power of two first, so neither large nor small ones leave fp32.
template <class T>
__global__ void __launch_bounds__(kThreads) norm_kernel(OrthoPlan p, Sources s, int64_t first, int64_t rows, int64_t cols,
                                                        int64_t ld) {
  after_previous();
  __shared__ float shared[kThreads / 32];
  const T* src = (const T*)s.p[blockIdx.y];
  const int64_t numel = rows * cols, turn = (int64_t)kThreads * kPerThread;
  double sum = 0.0;
  for (int64_t at = blockIdx.x * turn; at < numel; at += p.parts * turn) {
    float v[kPerThread], top = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
      const int64_t q = at + i * kThreads + threadIdx.x, r = q / cols;
      v[i] = q < numel ? element(src + r * ld + (q - r * cols)) : 0.0f;
      top = fmaxf(top, fabsf(v[i]));
      odd |= v[i] != v[i];
    }
    if (odd) top = CUDART_INF_F;
    top = reduce<true>(top, shared);
    if (top == 0.0f) continue;
    // 2^k, within the normal numbers
    const int k = top == CUDART_INF_F ? 0 : min(max(127 - (int)(__float_as_uint(top) >> 23), -126), 126);
    const float by = __uint_as_float((uint32_t)(127 + k) << 23);
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) part = fmaf(v[i] * by, v[i] * by, part);
    part = reduce<false>(part, shared);
    sum += ldexp((double)part, -2 * k);
  }
  if (threadIdx.x == 0) p.norms[(first + blockIdx.y) * p.parts + blockIdx.x] = sum;
}

// 1 / (norm + eps) as f 2^(i + j), f in [1, 2): each factor is one that fp32
// holds, whatever the norm.
struct Inverse {
  float f, i, j;
};
__device__ Inverse inverse_norm(const OrthoPlan& p, int64_t z, float eps) {
  double sum = 0.0;
  for (int q = 0; q < p.parts; ++q) sum += p.norms[z * p.parts + q];
  const double v = 1.0 / (sqrt(sum) + (double)eps);
  int e = 0;
  if (v == 0.0 || !(v < CUDART_INF)) return Inverse{(float)v, 1.0f, 1.0f};  // of infinity, 0 or NaN
  const double f = frexp(v, &e) * 2.0;
  e = min(max(e - 1, -240), 240);
  const int i = e / 2, j = e - i;
  return Inverse{(float)f, __uint_as_float((uint32_t)(127 + i) << 23), __uint_as_float((uint32_t)(127 + j) << 23)};
}

// The first X, 64 x 64 elements a CTA, turned where the matrix is tall.  With
// no steps to come it goes to the caller instead.
constexpr int kTile = 64;
template <class T>
__global__ void __launch_bounds__(kThreads) first_kernel(OrthoPlan p, Sources s, OrthoTargets out, int64_t first, int64_t rows,
                                                         int64_t cols, int64_t ld, float eps, float scale, int64_t ld_out) {
  after_previous();
  __shared__ float tile[kTile][kTile + 1];
  const int64_t z = first + blockIdx.y;
  const int64_t wide = (cols + kTile - 1) / kTile;
  const int64_t r0 = blockIdx.x / wide * kTile, c0 = blockIdx.x % wide * kTile;
  const T* src = (const T*)s.p[blockIdx.y];
  const Inverse inv = inverse_norm(p, z, eps);
  const int x = threadIdx.x % kTile, y0 = threadIdx.x / kTile;
  for (int y = y0; y < kTile; y += kThreads / kTile) {
    float v = 0.0f;
    if (r0 + y < rows && c0 + x < cols) v = element(src + (r0 + y) * ld + c0 + x) * inv.i * inv.f * inv.j;
    if (out.p[blockIdx.y]) {
      if (r0 + y < rows && c0 + x < cols) out.p[blockIdx.y][(r0 + y) * ld_out + c0 + x] = to_bf16(v);
      continue;
    }
    if (p.tall)
      tile[x][y] = v;
    else
      tile[y][x] = v;
  }
  if (out.p[blockIdx.y]) return;
  __syncthreads();
  const int64_t i0 = p.tall ? c0 : r0, j0 = p.tall ? r0 : c0;
  for (int y = y0; y < kTile; y += kThreads / kTile) {
    if (i0 + y >= p.m || j0 + x >= p.n) continue;
    const int64_t at = (z * p.m + i0 + y) * p.ld_x + j0 + x;
    split_half(tile[y][x] * scale, p.x[0][0][at], p.x[0][1][at]);
  }
}

// ------------------------------------------------------------ host side

int64_t line(int64_t v) { return (v + 63) / 64 * 64; }
int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

OrthoPlan plan_of(int64_t count, int64_t rows, int64_t cols, char* base, int64_t* bytes) {
  OrthoPlan p{};
  p.tall = rows > cols;
  p.m = (int)(p.tall ? cols : rows), p.n = (int)(p.tall ? rows : cols);
  p.count = count, p.ld_x = line(p.n), p.ld_a = line(p.m);
  const int64_t parts = ceil_div(rows * cols, (int64_t)kThreads * kPerThread);
  p.parts = (int)(parts < kMaxParts ? parts : kMaxParts);
  int64_t at = 0;
  const auto take = [&](int64_t n) {
    char* r = base + at;
    at += round256(n);
    return r;
  };
  for (auto& turn : p.x)
    for (auto& plane : turn) plane = (__half*)take(count * p.m * p.ld_x * 2);
  for (auto& plane : p.o) plane = (__half*)take(count * p.m * p.ld_a * 2);
  p.p = (__half*)take(count * p.m * p.ld_a * 2);
  p.d = (float*)take(count * p.m * 4), p.e = (float*)take(count * p.m * 4);
  p.norms = (double*)take(count * p.parts * 8);
  *bytes = at;
  return p;
}

// The largest magnitude of b x + c x x within [0, top].
double largest_b(double b, double c, double top) {
  double r = std::fabs(top * (b + c * top));
  const double x = -b / (2 * c);
  if (x > 0 && x < top) r = std::fmax(r, std::fabs(x * (b + c * x)));
  return r;
}
// And of s (a + b s^2 + c s^4).
double largest_x(double a, double b, double c, double top) {
  const auto f = [&](double s) { return std::fabs(s * (a + s * s * (b + c * s * s))); };
  double r = f(top);
  const double root = 9 * b * b - 20 * a * c;
  const double xs[3] = {(-3 * b + std::sqrt(root)) / (10 * c), (-3 * b - std::sqrt(root)) / (10 * c), -a / (3 * b)};
  for (double x : xs)  // NaN and infinities where there is no such place
    if (x > 0 && x < top * top) r = std::fmax(r, f(std::sqrt(x)));
  return r;
}

// The power of two that brings values up to `top` to 2^14 or below: a factor
// of 4 under fp16's largest.
double scale_for(double top) {
  int e = 0;
  std::frexp(std::fmax(top, 0x1p-30), &e);
  return std::ldexp(1.0, 14 - e);
}

// Each step's scales, from bounds of its matrices' norms; false where one
// passes 2^16.
bool steps_of(int steps, const float* k, OrthoStep* out) {
  double top = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = k[3 * i], b = k[3 * i + 1], c = k[3 * i + 2];
    const double next = largest_x(a, b, c, top);
    if (!(std::isfinite(a) && std::isfinite(b) && std::isfinite(c) && next <= 0x1p16)) return false;
    if (out)
      out[i] = OrthoStep{k[3 * i], k[3 * i + 1], k[3 * i + 2], (float)scale_for(top), (float)scale_for(top * top),
                         (float)scale_for(largest_b(b, c, top * top)), (float)scale_for(next)};
    top = next;
  }
  return true;
}

}  // namespace

int64_t ortho_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
  int64_t bytes = 0;
  plan_of(count, rows, cols, nullptr, &bytes);
  return bytes;
}

bool ortho_bounded(int steps, const float* coefficients) { return steps_of(steps, coefficients, nullptr); }

cudaError_t launch_orthogonalize(const OrthoArgs& a, const TcLaunch& l, cudaStream_t stream) {
  int64_t bytes = 0;
  const OrthoPlan p = plan_of(a.count, a.rows, a.cols, a.workspace, &bytes);
  OrthoStep steps[TIDE_MAX_ORTHOGONALIZE_STEPS] = {};
  if (!steps_of(a.steps, a.coefficients, steps)) return cudaErrorInvalidValue;
  const unsigned tiles = (unsigned)(ceil_div(a.rows, kTile) * ceil_div(a.cols, kTile));
  for (int64_t first = 0; first < a.count; first += kOrthoTable) {
    const unsigned some = (unsigned)(a.count - first < kOrthoTable ? a.count - first : kOrthoTable);
    Sources s{};
    OrthoTargets out{};
    for (unsigned i = 0; i < some; ++i) {
      s.p[i] = a.src[first + i];
      if (!a.steps) out.p[i] = a.dst[first + i];
    }
    cudaError_t e = launch_early(a.bf16 ? norm_kernel<uint16_t> : norm_kernel<float>, dim3(p.parts, some), kThreads, 0, 0,
                                 stream, p, s, first, a.rows, a.cols, a.ld_src);
    if (e == cudaSuccess)
      e = launch_early(a.bf16 ? first_kernel<uint16_t> : first_kernel<float>, dim3(tiles, some), kThreads, 0, 0, stream, p, s,
                       out, first, a.rows, a.cols, a.ld_src, a.eps, steps[0].x_scale, a.ld_dst);
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; i < a.steps; ++i)
    for (OrthoForm form : {kGram, kSquare, i + 1 < a.steps ? kUpdate : kLast}) {
      const cudaError_t e = launch_ortho_product(form, p, steps[i], i & 1, a, l, stream);
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace tide
