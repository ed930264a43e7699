// Newton-Schulz orthogonalisation: norms, the first X, short sides, and the steps.
//
// The first two kernels are passes over the matrices, bound by HBM: norms of
// one 14336 x 4096 in fp32 46 us (5.1 TB/s), its first X 112 (4.2; turned, and
// what was in L2 goes out meanwhile); 128 of 768 x 2048 in bf16 110 and 215 us.
#include <cmath>

#include "ortho.cuh"

namespace tide {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 1216;  // of all matrices, at most, whatever the device: the workspace holds as many

struct Sources {
  const void* p[kOrthoTable];
};

__device__ __forceinline__ float element(const float* p) { return *p; }
__device__ __forceinline__ float element(const uint16_t* p) { return bf16_value(*p); }

// V neighbours of a row, `left` of which there are; 0 past them.
template <int V, bool VEC, class T>
__device__ __forceinline__ void load_some(const T* p, int64_t left, float (&v)[V]) {
  if constexpr (VEC) {
    if (left >= V) {
      const uint4 q = *(const uint4*)p;
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4)
          v[i] = __uint_as_float(w[i]);
        else
          v[2 * i] = bf16_lo(w[i]), v[2 * i + 1] = bf16_hi(w[i]);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = i < left ? element(p + i) : 0.0f;
}

// A part of a matrix's sum of squares: a warp takes every so-manieth row.
// Elements whose squares might leave fp32 are brought near 1 by a power of
// two first; what they sum to is kept in 64 bits.  VEC: rows start on 16 bytes.
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) norm_kernel(OrthoPlan p, Sources s, int64_t first, int64_t rows, int64_t cols,
                                                        int64_t ld) {
  after_previous();
  constexpr int V = VEC ? 16 / sizeof(T) : 1;
  // loads of a lane on their way (with 4 of single elements three of 1021 x 1375
  // took 21 us instead of 9)
  constexpr int kFlight = VEC ? 4 : 16;
  __shared__ double shared[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  double sum = 0.0;
  for (int64_t r = (int64_t)blockIdx.x * kWarps + warp; r < rows; r += (int64_t)p.parts * kWarps) {
    const T* row = (const T*)s.p[blockIdx.y] + r * ld;
    for (int64_t c = 0; c < cols; c += 32 * V * kFlight) {
      float v[kFlight][V];
      uint32_t top = 0;  // of the magnitudes' bits: infinity and NaN above all
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        const int64_t at = c + (q * 32 + lane) * V;
        load_some<V, VEC>(row + at, cols - at, v[q]);
#pragma unroll
        for (int i = 0; i < V; ++i) top = max(top, __float_as_uint(v[q][i]) & 0x7fffffffu);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      const int e = (int)(top >> 23) - 127;
      const int k = e >= -40 && e <= 40 || top >= 0x7f800000u ? 0 : min(max(-e, -126), 126);
      const float by = __uint_as_float((uint32_t)(127 + k) << 23);
      float part = 0.0f;
#pragma unroll
      for (int q = 0; q < kFlight; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) part = fmaf(v[q][i] * by, v[q][i] * by, part);
      sum += k ? ldexp((double)part, -2 * k) : (double)part;
    }
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (lane == 0) shared[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) sum += shared[w];
    p.norms[(first + blockIdx.y) * p.parts + blockIdx.x] = sum;
  }
}

// 1 / (norm + eps) as f 2^(i + j): each factor is one that fp32 holds,
// whatever the norm.
struct Inverse {
  float f, i, j;
};
// 2^e, from the smallest normal number to the largest power.
__device__ __forceinline__ float power_of(int e) { return __uint_as_float((uint32_t)(127 + min(max(e, -126), 127)) << 23); }
// The sum is q 4^h, q in [1, 4): its root is taken in 32 bits, as 64-bit
// arithmetic would take longer than the kernel's loads.
__device__ __forceinline__ Inverse inverse_of(double sum, float eps) {
  // (a sum in 64 bits is infinite where an element is, and nowhere else)
  if (!(sum < CUDART_INF)) return Inverse{CUDART_NAN_F, 1.0f, 1.0f};
  const uint64_t b = (uint64_t)__double_as_longlong(sum);
  const int e = (int)(b >> 52) - 1023, h = e >> 1;
  float root = 0.0f;
  if (sum > 0.0) root = sqrtf(__double2float_rn(__longlong_as_double((int64_t)((b & 0xfffffffffffffull) | (uint64_t)(1023 + (e & 1)) << 52))));
  const int g = eps > 0.0f ? (int)(__float_as_uint(eps) >> 23) - 127 : -400;
  const int top = sum > 0.0 ? max(h, g) : g;
  // both over 2^top; where they are far apart the smaller one does not count
  const float norm = root * power_of(h - top) + (eps > 0.0f ? eps * power_of(-top) : 0.0f);
  const int i = -top / 2, j = -top - i;
  return Inverse{1.0f / norm, power_of(i), power_of(j)};
}
// One warp's, the parts in a fixed order: 64-bit sums of all warps would take
// longer (2048 x 2048: 10.4 us instead of 8.0).
__device__ __forceinline__ Inverse inverse_norm(const OrthoPlan& p, int64_t z, float eps) {
  __shared__ Inverse shared;
  if (threadIdx.x < 32) {
    double sum = 0.0;
#pragma unroll 8
    for (int q = threadIdx.x; q < p.parts; q += 32) sum += p.norms[z * p.parts + q];
    const int parts = min(p.parts, 32);
    for (int d = 1; d < parts; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (threadIdx.x == 0) shared = inverse_of(sum, eps);
  }
  __syncthreads();
  return shared;
}

// The first X, 64 x 64 elements a CTA, turned where the matrix is tall, 8
// neighbours of a row of X a thread.
constexpr int kTile = 64;
template <class T, bool VEC>
__global__ void __launch_bounds__(kThreads) first_kernel(OrthoPlan p, Sources s, int64_t first, int64_t rows, int64_t cols,
                                                         int64_t ld, int wide, float eps, float scale) {
  after_previous();
  constexpr int V = VEC ? 16 / sizeof(T) : 1;
  constexpr int kAcross = kTile / V, kPass = kThreads / kAcross, kPasses = kTile / kPass;
  __shared__ float tile[kTile][kTile + 1];
  const int64_t z = first + blockIdx.y;
  const int64_t r0 = (int64_t)(blockIdx.x / wide) * kTile, c0 = (int64_t)(blockIdx.x % wide) * kTile;
  const int x = threadIdx.x % kAcross * V, y0 = threadIdx.x / kAcross;
  const T* src = (const T*)s.p[blockIdx.y] + (r0 + y0) * ld + c0 + x;
  float v[kPasses][V];
#pragma unroll
  for (int q = 0; q < kPasses; ++q) {
    if (r0 + y0 + q * kPass < rows) {
      load_some<V, VEC>(src + q * kPass * ld, cols - c0 - x, v[q]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[q][i] = 0.0f;
    }
  }
  const Inverse inv = inverse_norm(p, z, eps);
#pragma unroll
  for (int q = 0; q < kPasses; ++q)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float f = v[q][i] * inv.i * inv.f * inv.j * scale;
      const int y = y0 + q * kPass;
      if (p.tall)
        tile[x + i][y] = f;
      else
        tile[y][x + i] = f;
    }
  __syncthreads();
  const int64_t i0 = p.tall ? c0 : r0, j0 = p.tall ? r0 : c0;
  const int xo = threadIdx.x % 8 * 8;
#pragma unroll
  for (int y = threadIdx.x / 8; y < kTile; y += kThreads / 8) {
    if (i0 + y >= p.m) continue;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) split_half2(tile[y][xo + 2 * i], tile[y][xo + 2 * i + 1], hi[i], lo[i]);
    // rows are whole 64s wide
    const int64_t at = (z * p.m + i0 + y) * p.ld_x + j0 + xo;
    *(uint4*)(p.x[0][0] + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *(uint4*)(p.x[0][1] + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}

// ------------------------------------------------------------ short sides

// Short sides of up to 16 rows: one fp16 term of a product's operands would
// leave 0.02 of the result next to rank one, and the products are too small for
// the tensor cores to matter.  X is kept in fp32, a CTA has a span of its columns: it
// adds up A from all spans' parts (in 64 bits, in order), makes C, takes its
// columns to C X, and leaves its part of the next A.  So a step is one launch, bound
// by what a launch and the parts' way take: one 8 x 4096 46 us (92 on the tensor
// cores, by pairs of steps), 64 of them 148 (163), 1000 of 16 x 64 298 (464).
constexpr int kShortTile = 64;  // columns at a time
// Of those a CTA, at least (one: 37 us and 243 for 64 of 8 x 4096, four: 61 and 131).
constexpr int kShortSpan = 2;

struct ShortStep {
  bool from_source, apply, last;  // no `apply`: A's first parts
  int turn;                       // of the parts that are written
  float a, b, c;
};

// The e-th pair i <= j of rows.
__device__ __forceinline__ void pair_of(int e, int m, int& i, int& j) {
  for (i = 0; e >= m - i; ++i) e -= m - i;
  j = i + e;
}

template <class T>
__global__ void __launch_bounds__(kThreads) short_kernel(OrthoPlan p, Sources s, OrthoTargets out, int64_t first, int64_t ld,
                                                         int64_t ld_out, float eps, ShortStep k) {
  after_previous();
  __shared__ float x[kShortSide][kShortTile + 1], y[kShortSide][kShortTile + 1];
  __shared__ float a[kShortSide][kShortSide + 1], c[kShortSide][kShortSide + 1];
  __shared__ double sums[kThreads];
  const int m = p.m, entries = m * (m + 1) / 2, slices = min(kThreads / entries, 32);
  const int64_t z = first + blockIdx.y;
  // an entry of A and a slice of what it is summed over
  const int entry = threadIdx.x % entries, slice = threadIdx.x / entries;
  int ei, ej;
  pair_of(entry, m, ei, ej);
  const auto add_up = [&](double v) {  // an entry's slices, in order: a sum for each of the first threads
    if (slice < slices) sums[threadIdx.x] = v;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x < entries)
      for (int q = 0; q < slices; ++q) sum += sums[q * entries + entry];
    __syncthreads();
    return sum;
  };
  if (k.apply) {
    const double* part = p.short_a[k.turn ^ 1] + z * p.spans * entries + entry;
    double v = 0.0;
    if (slice < slices)
#pragma unroll 8
      for (int q = slice; q < p.spans; q += slices) v += part[(int64_t)q * entries];
    const double sum = add_up(v);
    if (threadIdx.x < entries) a[ei][ej] = a[ej][ei] = (float)sum;
    __syncthreads();
    const int i = threadIdx.x / kShortSide, j = threadIdx.x % kShortSide;
    if (i < m && j < m) {
      float square = 0.0f;
      for (int q = 0; q < m; ++q) square = fmaf(a[i][q], a[q][j], square);
      c[i][j] = fmaf(k.c, square, fmaf(k.b, a[i][j], i == j ? k.a : 0.0f));
    }
    __syncthreads();
  }
  Inverse inv{};
  const T* src = (const T*)s.p[blockIdx.y];
  if (k.from_source) inv = inverse_norm(p, z, eps);
  float* const mine = p.short_x + z * m * p.ld_x;
  double all = 0.0;  // of this thread's entry and slice
  for (int n = 0; n < p.span; ++n) {
    const int64_t c0 = ((int64_t)blockIdx.x * p.span + n) * kShortTile;
    if (c0 >= p.n) break;
    for (int e = threadIdx.x; e < m * kShortTile; e += kThreads) {
      const bool turned = k.from_source && p.tall;
      const int i = turned ? e % m : e / kShortTile, q = turned ? e / m : e % kShortTile;
      const int64_t at = c0 + q;
      float v = 0.0f;
      if (at < p.n) {
        if (k.from_source)
          v = element(src + (p.tall ? at * ld + i : i * ld + at)) * inv.i * inv.f * inv.j;
        else
          v = mine[i * p.ld_x + at];
      }
      x[i][q] = v;
    }
    __syncthreads();
    if (k.apply) {
      for (int e = threadIdx.x; e < m * kShortTile; e += kThreads) {
        const int i = e / kShortTile, q = e % kShortTile;
        float v = 0.0f;
        for (int r = 0; r < m; ++r) v = fmaf(c[i][r], x[r][q], v);
        y[i][q] = v;
        if (!k.last && c0 + q < p.n) mine[i * p.ld_x + c0 + q] = v;
      }
      __syncthreads();
    }
    if (k.last) {
      uint16_t* to = out.p[blockIdx.y];
      for (int e = threadIdx.x; e < m * kShortTile; e += kThreads) {
        const int i = p.tall ? e % m : e / kShortTile, q = p.tall ? e / m : e % kShortTile;
        const int64_t at = c0 + q;
        if (at < p.n) to[p.tall ? at * ld_out + i : i * ld_out + at] = to_bf16(y[i][q]);
      }
    } else if (slice < slices) {
      const auto& t = k.apply ? y : x;
      float sum = 0.0f;
      for (int q = slice; q < kShortTile; q += slices) sum = fmaf(t[ei][q], t[ej][q], sum);
      all += sum;
    }
    __syncthreads();
  }
  if (k.last) return;
  const double sum = add_up(all);
  if (threadIdx.x < entries) p.short_a[k.turn][(z * p.spans + blockIdx.x) * entries + entry] = sum;
}

// A's planes of all segments, added up in their order: two neighbours of a row a
// thread, and its diagonal's element.  Each segment's rounding to fp16 is of its own
// size, so that all of them leave as much as A's own, about.
__global__ void __launch_bounds__(kThreads) join_kernel(OrthoPlan p, int out) {
  after_previous();
  const int64_t z = blockIdx.z, row = blockIdx.x, plane = (int64_t)p.m * p.ld_a;
  const int c = blockIdx.y * kThreads + threadIdx.x, pairs = (p.m + 1) / 2;
  if (c < pairs) {
    const __half* from = p.part_t + z * p.segments * plane + row * p.ld_a + 2 * c;
    float a = 0.0f, b = 0.0f;
#pragma unroll 8
    for (int s = 0; s < p.segments; ++s, from += plane) {
      const float2 v = __half22float2(*(const __half2*)from);
      a += v.x, b += v.y;
    }
    *(uint32_t*)(p.t[out] + z * plane + row * p.ld_a + 2 * c) = pack_half(a, b);
  } else if (c == pairs) {
    const float* from = p.part_d + z * p.segments * p.m + row;
    double sum = 0.0;
#pragma unroll 8
    for (int s = 0; s < p.segments; ++s, from += p.m) sum += *from;
    p.d[out][z * p.m + row] = (float)sum;
  }
}

// No steps: the normalised matrix itself.
template <class T>
__global__ void __launch_bounds__(kThreads) normalised_kernel(OrthoPlan p, Sources s, OrthoTargets out, int64_t first,
                                                              int64_t rows, int64_t cols, int64_t ld, int64_t ld_out, float eps) {
  after_previous();
  const T* src = (const T*)s.p[blockIdx.y];
  const Inverse inv = inverse_norm(p, first + blockIdx.y, eps);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += kThreads)
      out.p[blockIdx.y][r * ld_out + c] = to_bf16(element(src + r * ld + c) * inv.i * inv.f * inv.j);
}

// ------------------------------------------------------------ host side

int64_t line(int64_t v) { return (v + 63) / 64 * 64; }
int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

OrthoPlan plan_of(int64_t count, int64_t rows, int64_t cols, char* base, int64_t* bytes) {
  OrthoPlan p{};
  p.tall = rows > cols;
  p.m = (int)(p.tall ? cols : rows), p.n = (int)(p.tall ? rows : cols);
  p.count = count, p.ld_x = line(p.n), p.ld_a = line(p.m);
  // a row a warp, and no more CTAs than a device holds by and by (on 152 SMs
  // eight each)
  const int64_t room = ceil_div(kMaxParts, count), parts = ceil_div(rows, kWarps);
  p.parts = (int)(parts < room ? parts : room);
  int64_t at = 0;
  const auto take = [&](int64_t n) {
    char* r = base + at;
    at += round256(n);
    return r;
  };
  p.norms = (double*)take(count * p.parts * 8);
  if (p.m <= kShortSide) {
    // as many spans as the device has CTAs at a time, or, as each reads all spans'
    // parts, as those stay short; by the sizes alone, so that a matrix's sums are the
    // same among any number of others
    const int64_t tiles = ceil_div(p.n, kShortTile), entries = p.m * (p.m + 1) / 2;
    const int64_t most = 20000 / entries < kMaxParts ? 20000 / entries : kMaxParts;
    p.span = (int)ceil_div(tiles, most);
    if (p.span < kShortSpan) p.span = kShortSpan;
    p.spans = (int)ceil_div(tiles, p.span);
    p.short_x = (float*)take(count * p.m * p.ld_x * 4);
    for (auto& turn : p.short_a) turn = (double*)take(count * p.spans * entries * 8);
    *bytes = at;
    return p;
  }
  for (auto& turn : p.x)
    for (auto& plane : turn) plane = (__half*)take(count * p.m * p.ld_x * 2);
  for (auto& plane : p.t) plane = (__half*)take(count * p.m * p.ld_a * 2);
  for (auto& diagonal : p.d) diagonal = (float*)take(count * p.m * 4);
  p.x_terms = p.m <= 64 ? 2 : 1;
  p.segments = (int)ceil_div(p.n, kOrthoSegment);
  if (p.segments > 1) {
    p.part_t = (__half*)take(count * p.segments * p.m * p.ld_a * 2);
    p.part_d = (float*)take(count * p.segments * p.m * 4);
  }
  *bytes = at;
  return p;
}

// The largest magnitude of a + b x + c x x within [0, top].
double largest_c(double a, double b, double c, double top) {
  const auto f = [&](double x) { return std::fabs(a + x * (b + c * x)); };
  const double x = -b / (2 * c);  // NaN or infinity where there is no such place
  const double r = std::fmax(f(0), f(top));
  return x > 0 && x < top ? std::fmax(r, f(x)) : r;
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

// Bounds of norms: of each step's X, and of its C.
struct Bounds {
  double x[TIDE_MAX_ORTHOGONALIZE_STEPS + 1], c[TIDE_MAX_ORTHOGONALIZE_STEPS];
};
// False where one of X passes 2^16.
bool bounds_of(int steps, const float* k, Bounds* out) {
  out->x[0] = 1.0;
  for (int i = 0; i < steps; ++i) {
    const double a = k[3 * i], b = k[3 * i + 1], c = k[3 * i + 2], top = out->x[i];
    out->x[i + 1] = largest_x(a, b, c, top);
    out->c[i] = largest_c(a, b, c, top * top);
    if (!(std::isfinite(a) && std::isfinite(b) && std::isfinite(c) && out->x[i + 1] <= 0x1p16)) return false;
  }
  return true;
}

// Whether step i and the next share a pass over X: 5 products of m^3 / 2
// operations and 3 of m m n / 2 instead of 2 and 6.  An error of A grows by up
// to a^2 on its way to the second step's, which a moderate a only allows; it
// leaves less the more rows there are (ortho.cuh).  So steps share a pass where it
// pays: 14336 x 4096 takes 2.18 ms instead of 2.79 by single steps, four of 2048 x
// 8192 1.26 instead of 1.66, 128 of 768 x 2048 2.56 instead of 2.99, eight of 600 x
// 2400 247 us instead of 286; of two sides that are nearer to one another or shorter
// they save less than 5% (64 of 1024 x 1536 1.85 ms and 1.91, 384 x 1024 99 us and
// 104, 512 x 2048 122 and 117), but for thin ones (27 of 3131 x 257 385 us and 482,
// 3457 x 63 100 and 121, 128 x 2048 84 and 94).
constexpr int kPairedSide = 384;
bool paired(const OrthoPlan& p, const OrthoArgs& a, int i) {
  const float k = a.coefficients[3 * i];
  return i + 1 < a.steps && p.m >= kPairedSide && 2 * (int64_t)p.n >= 5 * (int64_t)p.m && k * k <= 16.0f;
}

// How far steps from i on may stretch what is small.
float stretch_from(const OrthoArgs& a, int i) {
  float r = 1.0f;
  for (; i < a.steps; ++i) r *= std::fabs(a.coefficients[3 * i]);
  return r;
}

}  // namespace

cudaError_t launch_ortho_join(const OrthoPlan& p, int out, cudaStream_t stream) {
  const unsigned across = (unsigned)ceil_div((p.m + 1) / 2 + 1, kThreads);
  OrthoPlan k = p;
  for (int64_t z = 0; z < p.count; z += kOrthoTable) {
    const unsigned some = (unsigned)(p.count - z < kOrthoTable ? p.count - z : kOrthoTable);
    k.part_t = p.part_t + z * p.segments * p.m * p.ld_a, k.part_d = p.part_d + z * p.segments * p.m;
    k.t[out] = p.t[out] + z * p.m * p.ld_a, k.d[out] = p.d[out] + z * p.m;
    const cudaError_t e = launch_early(join_kernel, dim3((unsigned)p.m, across, some), kThreads, 0, 0, stream, k, out);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int64_t ortho_workspace_bytes(int64_t count, int64_t rows, int64_t cols) {
  int64_t bytes = 0;
  plan_of(count, rows, cols, nullptr, &bytes);
  return bytes;
}

bool ortho_bounded(int steps, const float* coefficients) {
  Bounds b;
  return bounds_of(steps, coefficients, &b);
}

cudaError_t launch_orthogonalize(const OrthoArgs& a, const TcLaunch& l, cudaStream_t stream) {
  int64_t bytes = 0;
  const OrthoPlan p = plan_of(a.count, a.rows, a.cols, a.workspace, &bytes);
  Bounds bound;
  if (!bounds_of(a.steps, a.coefficients, &bound)) return cudaErrorInvalidValue;
  const int64_t wide = ceil_div(a.cols, kTile), tiles = ceil_div(a.rows, kTile) * wide;
  for (int64_t first = 0; first < a.count; first += kOrthoTable) {
    const unsigned some = (unsigned)(a.count - first < kOrthoTable ? a.count - first : kOrthoTable);
    Sources s{};
    OrthoTargets out{};
    bool vec = a.ld_src % (a.bf16 ? 8 : 4) == 0;
    for (unsigned i = 0; i < some; ++i) {
      s.p[i] = a.src[first + i];
      vec = vec && (uintptr_t)s.p[i] % 16 == 0;
      out.p[i] = a.dst[first + i];
    }
    cudaError_t e = launch_early(a.bf16 ? vec ? norm_kernel<uint16_t, true> : norm_kernel<uint16_t, false>
                                 : vec  ? norm_kernel<float, true>
                                        : norm_kernel<float, false>,
                                 dim3(p.parts, some), kThreads, 0, 0, stream, p, s, first, a.rows, a.cols, a.ld_src);
    if (p.m <= kShortSide && a.steps) {
      for (int i = -1; i < a.steps && e == cudaSuccess; ++i) {  // A's first parts, then the steps
        const float* c = a.coefficients + 3 * (i < 0 ? 0 : i);
        e = launch_early(a.bf16 ? short_kernel<uint16_t> : short_kernel<float>, dim3(p.spans, some), kThreads, 0, 0, stream, p, s, out,
                         first, a.ld_src, a.ld_dst, a.eps, ShortStep{i <= 0, i >= 0, i == a.steps - 1, i & 1, c[0], c[1], c[2]});
      }
    } else if (e == cudaSuccess && a.steps)
      e = launch_early(a.bf16 ? vec ? first_kernel<uint16_t, true> : first_kernel<uint16_t, false>
                       : vec  ? first_kernel<float, true>
                              : first_kernel<float, false>,
                       dim3((unsigned)tiles, some), kThreads, 0, 0, stream, p, s, first, a.rows, a.cols, a.ld_src, (int)wide,
                       a.eps, (float)scale_for(1.0));
    else if (e == cudaSuccess)
      e = launch_early(a.bf16 ? normalised_kernel<uint16_t> : normalised_kernel<float>,
                       dim3((unsigned)(a.rows < 4096 ? a.rows : 4096), some), kThreads, 0, 0, stream, p, s, out, first, a.rows,
                       a.cols, a.ld_src, a.ld_dst, a.eps);
    if (e != cudaSuccess) return e;
  }
  if (!a.steps || p.m <= kShortSide) return cudaSuccess;
  OrthoProduct q[4 * TIDE_MAX_ORTHOGONALIZE_STEPS];  // 3 a step, 7 for two that share a pass
  int products = 0, turn = 0;
  for (int i = 0; i < a.steps; turn ^= 1) {
    const bool two = paired(p, a, i);
    const float x = (float)scale_for(bound.x[i]);
    float t[3] = {};  // scales of what lies in the symmetric places
    const auto sym = [&](int left, int right, int out, double top, float s2, float s1, float s0) {
      const float scale = (float)scale_for(top);
      q[products++] = OrthoProduct{kSym, turn, left, right, out, s2, s1, s0, t[left], t[right], scale, 0};
      t[out] = scale;
    };
    const auto square = [&](int from, int out, int step) {
      const float* k = a.coefficients + 3 * step;
      sym(from, from, out, bound.c[step], k[2], k[1], k[0]);
    };
    t[0] = (float)scale_for(bound.x[i] * bound.x[i]);
    q[products++] = OrthoProduct{kGram, turn, 0, 0, 0, 1, 0, 0, x, x, t[0], 0};
    square(0, 1, i);  // C
    if (two) {
      sym(1, 0, 2, bound.c[i] * bound.x[i] * bound.x[i], 1, 0, 0);  // C A
      sym(2, 1, 0, bound.x[i + 1] * bound.x[i + 1], 1, 0, 0);       // C A C: the next A
      square(0, 2, i + 1);                                          // C'
      sym(2, 1, 0, bound.c[i] * bound.c[i + 1], 1, 0, 0);           // C' C
    }
    const float first = a.coefficients[3 * i] * (two ? a.coefficients[3 * i + 3] : 1.0f);  // L(0)
    i += two ? 2 : 1;
    const int by = two ? 0 : 1;
    const float rest = p.x_terms == 1 && stretch_from(a, i) > 8.0f ? first : 0.0f;
    q[products++] =
        OrthoProduct{i < a.steps ? kUpdate : kLast, turn, 0, by, 0, 1, 0, 0, x, t[by], (float)scale_for(bound.x[i]), rest};
  }
  return launch_ortho_products(p, q, products, a, l, stream);
}

}  // namespace tide
