// Routing of tokens to experts, its backward pass, and the experts' order.
//
// A warp takes a token: each lane holds a run of neighbouring experts' logits
// in registers, so nothing is read twice and, as the lowest lane holds the
// lowest indices, equals go to the lowest index by going to the lowest lane.
// Bound by instructions, some 1,400 a token of 256 experts in groups (8192 of
// them 16 to 18 us, of 128 experts without 7, backward 5), and by the few tokens
// whose borders take 64 bits (33 us with all of a token's scores in them).
#include "compute_device.cuh"

namespace tide {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;

template <class T>
__device__ __forceinline__ float value_of(const T* p);
template <>
__device__ __forceinline__ float value_of(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float value_of(const uint16_t* p) {
  return bf16_value(*p);
}

// A row's logits, `own` a lane from its first on; -infinity past the end.
// VEC: rows start on 16 bytes and a lane's run is whole 16-byte (or 8-byte)
// vectors.
template <int N, bool VEC, class T>
__device__ __forceinline__ void load_row(const T* row, int first, int own, int experts, float (&l)[N]) {
  if constexpr (VEC) {
    constexpr int kEach = 4;  // 16 bytes of fp32, 8 of bf16
#pragma unroll
    for (int i = 0; i < N; i += kEach) {
      float v[kEach];
#pragma unroll
      for (int q = 0; q < kEach; ++q) v[q] = -CUDART_INF_F;
      if (i < own && first + i < experts) {
        if constexpr (sizeof(T) == 4) {
          const float4 f = *(const float4*)(row + first + i);
          v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
          const uint2 f = *(const uint2*)(row + first + i);
          v[0] = bf16_lo(f.x), v[1] = bf16_hi(f.x), v[2] = bf16_lo(f.y), v[3] = bf16_hi(f.y);
        }
      }
#pragma unroll
      for (int q = 0; q < kEach; ++q) l[i + q] = v[q];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      l[i] = i < own && first + i < experts ? value_of(row + first + i) : -CUDART_INF_F;
  }
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
template <class F>
__device__ __forceinline__ F warp_sum(F v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Whole numbers in the order of the values: 0 for what cannot be chosen, 1
// for NaN, then from -infinity on; both zeros are the same.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return v != v ? 1u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t key_of(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return v != v ? 1ull : b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float value_of_key(uint32_t k) {
  return k <= 1u ? CUDART_NAN_F : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ double value_of_key(uint64_t k) {
  return k <= 1u ? CUDART_NAN : __longlong_as_double((int64_t)(k >> 63 ? k ^ 0x8000000000000000ull : ~k));
}
__device__ __forceinline__ uint32_t max_key(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t max_key(uint64_t k) {
  const uint32_t hi = max_key((uint32_t)(k >> 32));
  const uint32_t lo = max_key((uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// The scores of a lane's run.  Softmax: top is the row's largest logit; a row
// of masked experts has scores of 0.
template <int N>
__device__ __forceinline__ void scores_of(const float (&l)[N], bool sigmoid, float top, float (&s)[N]) {
  if (sigmoid) {
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = 1.0f / (1.0f + expf(-l[i]));
    return;
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = top == -CUDART_INF_F && l[i] == top ? 0.0f : expf(l[i] - top);
    sum += s[i];
  }
  sum = warp_sum(sum);
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = sum == 0.0f ? 0.0f : s[i] / sum;
}

// What a router's choice needs of its arguments.
struct Choice {
  int experts, own, topk, groups, each, top_groups, group_best;
  int lanes;  // of a group, if groups are whole lanes' runs and those a power of two; else 0
};

// What a group's score is made of, by magnitude: its rounding goes by that,
// whatever the terms come to (two of opposite signs leave theirs in a small
// sum).  Nothing where a term is infinite or NaN, which no rounding moves.
template <class F>
__device__ __forceinline__ float reach_of(F best, F next) {
  const F top = F(CUDART_INF_F);
  return fabs(best) < top && fabs(next) < top ? (float)(fabs(best) + fabs(next)) : 0.0f;
}

// Drops the keys of groups that are not among the best.  Returns whether the
// groups on either side of the border are no further apart than `near` times
// (1 + twice the largest magnitude of any group's terms), which two scores'
// roundings stay below; then nothing is dropped.  `second` receives the key
// that a group's score goes down to, where a group is whole lanes.
template <int N, class K>
__device__ __forceinline__ bool keep_groups(const Choice& c, int first, float near, K (&key)[N], K* second = nullptr) {
  using F = decltype(value_of_key(K()));
  const int lane = threadIdx.x & 31;
  // Lane g's score of group g, or, where a group is whole lanes, each lane's
  // of its own group.
  K order;
  float reach = 0.0f;
  if (c.lanes) {
    K best = 0, next = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const K k = key[i];
      next = max(next, min(best, k));
      best = max(best, k);
    }
    for (int d = 1; d < c.lanes; d <<= 1) {
      const K b = __shfl_xor_sync(0xffffffffu, best, d), n = __shfl_xor_sync(0xffffffffu, next, d);
      next = max(max(next, n), min(best, b));
      best = max(best, b);
    }
    F score = value_of_key(best);
    const bool two = c.group_best == 2 && c.each > 1;
    const F rest = two ? value_of_key(next) : F(0);
    reach = reach_of(score, rest);
    if (two) score += rest;
    order = key_of(score);
    if (second) *second = two ? next : best;
  } else {
    F mine = 0;
    for (int g = 0; g < c.groups; ++g) {
      const int lo = g * c.each - first, hi = lo + c.each;  // the group among this lane's run
      K best = 0, next = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const K k = i >= lo && i < hi ? key[i] : 0;
        next = max(next, min(best, k));
        best = max(best, k);
      }
      const K top = max_key(best);
      F score = value_of_key(top), rest = 0;
      if (c.group_best == 2 && c.each > 1) {
        const int owner = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        rest = value_of_key(max_key(lane == owner ? next : best));
      }
      reach = fmaxf(reach, reach_of(score, rest));
      if (c.group_best == 2 && c.each > 1) score += rest;
      if (lane == g) mine = score;
    }
    order = lane < c.groups ? key_of(mine) : 0;
  }
  const int step = c.lanes ? c.lanes : 1, me = lane / step;
  int above = 0;
  for (int g = 0; g < c.groups; ++g) {
    const K other = __shfl_sync(0xffffffffu, order, g * step);
    above += other > order || (other == order && g < me);
  }
  const bool in = me < c.groups, stays = in && above < c.top_groups;
  if (near > 0.0f && c.top_groups < c.groups) {
    // the border: the lowest kept, the highest left
    const K low = (K)~max_key((K)~(stays ? order : (K)~(K)0)), high = max_key(in && !stays ? order : (K)0);
    const F a = value_of_key(low), b = value_of_key(high);
    reach = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(reach)));
    // (scores that leave fp32, but whose terms do not, are as good as equal here)
    if (reach == CUDART_INF_F) return true;
    const bool close = a - b <= F(near) * (F(1) + F(2) * F(reach)) && fabs(a) < F(CUDART_INF_F) && fabs(b) < F(CUDART_INF_F);
    if (close) return true;
  }
  const uint32_t kept = __ballot_sync(0xffffffffu, stays);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (!(c.lanes ? stays : (bool)(kept >> min((first + i) / c.each, 31) & 1))) key[i] = 0;
  return false;
}

// The largest keys in order, from the `from`-th to before the `to`-th: lane j
// returns the j-th's expert and its key, other lanes what they had.
template <int N, class K>
__device__ __forceinline__ int pick(const Choice& c, int first, int from, int to, K (&key)[N], int mine, K* picked) {
  const int lane = threadIdx.x & 31;
  for (int j = from; j < to; ++j) {
    K best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key[i] > best) best = key[i], at = i;
    const K top = max_key(best);
    const int owner = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
    const int expert = __shfl_sync(0xffffffffu, first + at, owner);
    if (lane == j) mine = expert, *picked = top;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane == owner && i == at) key[i] = 0;
  }
  return mine;
}
template <int N, class K>
__device__ __forceinline__ int pick(const Choice& c, int first, K (&key)[N]) {
  K picked = 0;
  return pick(c, first, 0, c.topk, key, 0, &picked);
}

// A lane's weight from its pick's logit, before the scale.  With
// renormalisation a softmax goes by the picks alone; so do sigmoids where one of
// the picks is far below zero, where a sigmoid is exp(l) to fp32's last bit and
// may itself be below what fp32 holds, though its share is not: e^-top s for top
// up to 0, as exp(l - top) / (1 + exp(l)).
__device__ __forceinline__ float weight_of(float l, bool in, bool sigmoid, bool renormalize, float score) {
  if (!renormalize) return score;
  const float top = warp_max(in ? l : -CUDART_INF_F);
  float s = score;
  if (!sigmoid) {
    s = top == -CUDART_INF_F && l == top ? 0.0f : expf(l - top);
  } else if (__any_sync(0xffffffffu, in && l < -60.0f)) {
    const float from = fminf(top, 0.0f);
    if (l <= 0.0f) s = l == -CUDART_INF_F ? 0.0f : expf(l - from) / (1.0f + expf(l));
  }
  if (!in) s = 0.0f;
  const float sum = warp_sum(s);
  return sum == 0.0f ? 0.0f : s / sum;
}

// The sum of a softmax's exponentials in 64 bits, several on their way at a
// time: one by one they took 17 us of a call's 31.
template <int N>
__device__ __noinline__ double wide_sum(const float (&l)[N], float top) {
  double sum = 0.0;
#pragma unroll(N < 8 ? N : 8)
  for (int i = 0; i < N; ++i) {
    const double e = exp((double)l[i] - (double)top);
    sum += top == -CUDART_INF_F && l[i] == top ? 0.0 : e;
  }
  return warp_sum(sum);
}
// A score plus bias in 64 bits.
__device__ __noinline__ double wide_choice(float l, float bias, bool sigmoid, float top, double sum) {
  double s = 0.0;
  if (sigmoid)
    s = 1.0 / (1.0 + exp(-(double)l));
  else if (sum != 0.0 && l != -CUDART_INF_F)
    s = exp((double)l - (double)top) / sum;
  return s + (double)bias;
}

// Keys in 64 bits of what may count: all whose key in 32 is at least `from`.
template <int N>
__device__ __noinline__ void wide_keys(const Choice& c, int first, const float (&l)[N], const uint32_t (&key)[N], uint32_t from,
                                       bool sigmoid, float top, const float* bias, uint64_t (&wide)[N]) {
  const double sum = sigmoid ? 0.0 : wide_sum(l, top);
  // a lane's own ones after another, not the places of all lanes'
  uint32_t left = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    wide[i] = 0;
    left |= (key[i] && key[i] >= from ? 1u : 0u) << i;
  }
  while (left) {
    const int i = __ffs(left) - 1;
    left &= left - 1;
    wide[i] = key_of(wide_choice(l[i], bias ? bias[first + i] : 0.0f, sigmoid, top, sum));
  }
  __syncwarp();
}

// Drops groups by their scores in 64 bits.  Where a group is whole lanes,
// only what may be among its best two is looked at: few a lane.
template <int N>
__device__ __noinline__ void keep_groups_wide(const Choice& c, int first, const float (&l)[N], uint32_t second, float near,
                                              bool sigmoid, float top, const float* bias, uint32_t (&key)[N]) {
  uint64_t wide[N];
  uint32_t from = 1;
  if (c.lanes) {
    const float v = value_of_key(second);
    from = fabsf(v) < CUDART_INF_F ? key_of(v - near * (1.0f + fabsf(v))) : second;
  }
  wide_keys(c, first, l, key, from, sigmoid, top, bias, wide);
  keep_groups(c, first, 0.0f, wide);
  // a kept group has its best ones' keys; what was not looked at goes with them
  bool stays = false;
#pragma unroll
  for (int i = 0; i < N; ++i) stays |= wide[i] != 0;
  for (int d = 1; d < c.lanes; d <<= 1) stays |= __shfl_xor_sync(0xffffffffu, (int)stays, d) != 0;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (c.lanes ? !stays : !wide[i]) key[i] = 0;
}

// N: logits a lane holds, at least ceil(experts / 32).
template <int N, bool VEC, class T>
__global__ void __launch_bounds__(kThreads) route_kernel(RouterArgs a, Choice c) {
  after_previous();
  const int lane = threadIdx.x & 31, first = lane * c.own;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const bool sigmoid = a.score == TIDE_SCORE_SIGMOID;
  const T* row = (const T*)a.logits + t * a.ld;
  float l[N];
  load_row<N, VEC>(row, first, c.own, c.experts, l);
  float top = -CUDART_INF_F;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, l[i]), nan |= l[i] != l[i];
  top = warp_max(top);
  nan = __any_sync(0xffffffffu, nan);

  // Scores grow with logits, so without a bias logits decide, exactly.
  const bool direct = !a.bias && (c.groups == 1 || c.group_best == 1 || c.each == 1);
  float sum = 0.0f;
  int expert;
  if (direct) {
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) key[i] = i < c.own && first + i < c.experts ? key_of(l[i]) : 0;
    if (c.groups > 1) keep_groups(c, first, 0.0f, key);
    expert = pick(c, first, key);
  } else {
    float s[N];
    uint32_t key[N], picked;
    scores_of(l, sigmoid, top, s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = i < c.own && first + i < c.experts;
      key[i] = in ? key_of(s[i] + (a.bias ? a.bias[first + i] : 0.0f)) : 0;
    }
    // A sigmoid here is off by at most 4 2^-24 of itself, a softmax by 64
    // (its sum of up to 1024 terms 37 of them), a sum with the bias by 2^-24
    // of itself more.  So `near` is how far apart any two of a row may seem
    // that are equal, with as much again; what is further apart is in order.
    float near = 0x1p-20f;
    if (!sigmoid) {
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < N; ++i) most = fmaxf(most, s[i]);
      near = 0x1p-16f * warp_max(most);
    }
    if (c.groups > 1) {
      const float apart = sigmoid ? 0x1p-20f : 0x1p-16f;
      uint32_t second = 0;
      if (keep_groups(c, first, apart, key, &second)) keep_groups_wide(c, first, l, second, apart, sigmoid, top, a.bias, key);
    }
    uint32_t allowed = 0;  // of this lane's run
#pragma unroll
    for (int i = 0; i < N; ++i) allowed |= (key[i] != 0 ? 1u : 0u) << i;
    // more than are wanted, as long as the last one's neighbour may be before it
    int rounds = min(c.topk + 1, c.experts), at = 0;
    expert = 0, picked = 0;
    bool close = false;
    while (true) {
      expert = pick(c, first, at, rounds, key, expert, &picked);
      const float mine = value_of_key(picked);
      const float b = a.bias && lane < rounds ? a.bias[expert] : 0.0f, l0 = lane < rounds ? value_of(row + expert) : 0.0f;
      const float next = __shfl_down_sync(0xffffffffu, mine, 1), next_b = __shfl_down_sync(0xffffffffu, b, 1);
      const float next_l = __shfl_down_sync(0xffffffffu, l0, 1);
      const uint32_t next_key = __shfl_down_sync(0xffffffffu, picked, 1);
      const bool pair = lane + 1 < rounds && next_key > 1u && fabsf(mine) < CUDART_INF_F && fabsf(next) < CUDART_INF_F;
      // equal logits with equal biases are equals, whatever the rounding
      const bool equal = pair && l0 == next_l && b == next_b;
      const uint32_t equals = __ballot_sync(0xffffffffu, equal);
      const uint32_t which = __ballot_sync(0xffffffffu, pair && !equal && mine - next <= near + 0x1p-22f * (fabsf(mine) + fabsf(next)));
      close = which != 0;
      if (rounds < 2 || rounds >= min(c.experts, 32) || !((which | equals) >> (rounds - 2) & 1)) break;
      at = rounds++;
    }
    if (close) {
      if (rounds == 32 && c.experts > 32) {  // more than a warp holds: all of them again
        uint64_t wide[N];
        uint32_t all[N];
#pragma unroll
        for (int i = 0; i < N; ++i) all[i] = allowed >> i & 1;
        wide_keys(c, first, l, all, 1, sigmoid, top, a.bias, wide);
        expert = pick(c, first, wide);
      } else {
        const double sum = sigmoid ? 0.0 : wide_sum(l, top);
        // the picks again, by 64 bits; what cannot be chosen stays last
        const float b = a.bias ? a.bias[expert] : 0.0f;
        uint64_t order = 0;
        if (lane < rounds && picked) order = key_of(wide_choice(value_of(row + expert), b, sigmoid, top, sum));
        int rank = 0;
        for (int j = 0; j < rounds; ++j) {
          const uint64_t other = __shfl_sync(0xffffffffu, order, j);
          const int e = __shfl_sync(0xffffffffu, expert, j);
          rank += other > order || (other == order && e < expert);
        }
        int mine = expert;
        for (int j = 0; j < rounds; ++j) {
          const int r = __shfl_sync(0xffffffffu, rank, j), e = __shfl_sync(0xffffffffu, expert, j);
          if (r == lane) mine = e;
        }
        expert = mine;
      }
    }
  }
  if (!sigmoid && !a.renormalize) {
#pragma unroll
    for (int i = 0; i < N; ++i) sum += top == -CUDART_INF_F && l[i] == top ? 0.0f : expf(l[i] - top);
    sum = warp_sum(sum);
  }
  const bool in = lane < c.topk;
  const float mine = in ? value_of(row + expert) : 0.0f;
  float score;
  if (sigmoid)
    score = 1.0f / (1.0f + expf(-mine));
  else
    score = sum == 0.0f || mine == -CUDART_INF_F ? 0.0f : expf(mine - top) / sum;
  float w = weight_of(mine, in, sigmoid, a.renormalize, score) * a.scale;
  if (!sigmoid && (nan || top == CUDART_INF_F)) w = CUDART_NAN_F;
  if (in) {
    a.ids[t * c.topk + lane] = expert;
    a.weights[t * c.topk + lane] = w;
  }
}

// dl = s (g - sum g s) over a softmax; s (1 - s) g of a sigmoid; with
// renormalisation p (g - sum g p), p the weights before the scale, times (1 -
// s) of a sigmoid, over the picks alone.
template <int N, bool VEC, class T>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(RouterArgs a, Choice c) {
  after_previous();
  const int lane = threadIdx.x & 31, first = lane * c.own;
  const int64_t t = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const bool sigmoid = a.score == TIDE_SCORE_SIGMOID;
  const T* row = (const T*)a.logits + t * a.ld;
  int id = -1;
  float g = 0.0f;
  if (lane < c.topk) id = a.ids[t * c.topk + lane], g = a.dweights[t * c.topk + lane] * a.scale;
  const bool in = (unsigned)id < (unsigned)c.experts;
  if (!in) g = 0.0f;
  const float mine = in ? value_of(row + id) : -CUDART_INF_F;
  float d[N];  // of this lane's run
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = 0.0f;
  float dl = g;  // of this lane's pick
  const bool whole = !sigmoid && !a.renormalize;
  if (!whole) {
    const float s = 1.0f / (1.0f + expf(-mine)), rest = 1.0f / (1.0f + expf(mine));
    const float p = weight_of(mine, in, sigmoid, a.renormalize, s);
    if (a.renormalize) {
      const float mean = warp_sum(in ? p * g : 0.0f);
      dl = p * (g - mean) * (sigmoid ? rest : 1.0f);
    } else {
      dl = g * s * rest;
    }
  }
  for (int j = 0; j < c.topk; ++j) {
    const int e = __shfl_sync(0xffffffffu, id, j) - first;
    const float v = __shfl_sync(0xffffffffu, dl, j);
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (e == i && i < c.own) d[i] += v;
  }
  if (whole) {
    float l[N], s[N], top = -CUDART_INF_F, mean = 0.0f;
    load_row<N, VEC>(row, first, c.own, c.experts, l);
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, l[i]);
    scores_of(l, false, warp_max(top), s);
#pragma unroll
    for (int i = 0; i < N; ++i) mean += d[i] * s[i];
    mean = warp_sum(mean);
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = s[i] * (d[i] - mean);
  }
  T* out = (T*)a.dlogits + t * a.ldd;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      if (i < c.own && first + i < c.experts) {
        if constexpr (sizeof(T) == 4)
          *(float4*)(out + first + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
        else
          *(uint2*)(out + first + i) = make_uint2(pack_bf16(d[i], d[i + 1]), pack_bf16(d[i + 2], d[i + 3]));
      }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < c.own && first + i < c.experts) {
        if constexpr (sizeof(T) == 4)
          out[first + i] = d[i];
        else
          out[first + i] = to_bf16(d[i]);
      }
  }
}

enum Pass { kForward, kBackward };

template <Pass P, int N, class T>
cudaError_t run(const RouterArgs& a, const Choice& c, bool vec, cudaStream_t stream) {
  const dim3 grid((unsigned)ceil_div(a.tokens, kWarps));
  if constexpr (N % 4 == 0) {
    if (vec)
      return P == kForward ? launch_early(route_kernel<N, true, T>, grid, kThreads, 0, 0, stream, a, c)
                           : launch_early(route_backward_kernel<N, true, T>, grid, kThreads, 0, 0, stream, a, c);
  }
  return P == kForward ? launch_early(route_kernel<N, false, T>, grid, kThreads, 0, 0, stream, a, c)
                       : launch_early(route_backward_kernel<N, false, T>, grid, kThreads, 0, 0, stream, a, c);
}

template <Pass P, class T>
cudaError_t run(const RouterArgs& a, cudaStream_t stream) {
  const int own = (int)ceil_div(a.experts, 32);
  const int each = a.experts / a.groups, lanes = each / own;
  const Choice c{a.experts, own, a.topk, a.groups, each, a.top_groups, a.group_best,
                 each % own == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0};
  const auto whole = [](const void* p, int64_t ld) { return (uintptr_t)p % (4 * sizeof(T)) == 0 && ld % 4 == 0; };
  const bool vec = own % 4 == 0 && a.experts % 4 == 0 && whole(a.logits, a.ld) && (P == kForward || whole(a.dlogits, a.ldd));
  if (own <= 1) return run<P, 1, T>(a, c, vec, stream);
  if (own <= 2) return run<P, 2, T>(a, c, vec, stream);
  if (own <= 4) return run<P, 4, T>(a, c, vec, stream);
  if (own <= 8) return run<P, 8, T>(a, c, vec, stream);
  if (own <= 16) return run<P, 16, T>(a, c, vec, stream);
  return run<P, 32, T>(a, c, vec, stream);
}

// ------------------------------------------------------- the experts' order

constexpr int kSlotWarps = 8;
constexpr int kSlotThreads = 32 * kSlotWarps;
constexpr int kChunk = 1024;      // pairs of a CTA, at least
constexpr int kMaxChunks = 304;

int64_t chunk_of(int64_t pairs) {
  const int64_t least = ceil_div(pairs, kMaxChunks);
  return least <= kChunk ? kChunk : ceil_div(least, kSlotThreads) * kSlotThreads;
}

// How many of each chunk's pairs each expert has.
__global__ void __launch_bounds__(kSlotThreads) count_kernel(SlotsArgs a, int64_t chunk) {
  after_previous();
  __shared__ int count[TIDE_MAX_EXPERTS];
  for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) count[e] = 0;
  __syncthreads();
  const int64_t from = blockIdx.x * chunk, to = min(a.pairs, from + chunk);
  for (int64_t i = from + threadIdx.x; i < to; i += kSlotThreads) {
    const int e = a.ids[i];
    if ((unsigned)e < (unsigned)a.experts) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSlotThreads) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// Each pair's place (65,528 pairs of 128 experts: 7 us, the counts before them
// 2.5).  A CTA finds where its chunk's pairs of each expert begin
// (the experts before, and this expert's in the chunks before), each warp
// where its own run's do, and goes through that run 32 pairs at a time:
// whole numbers throughout, so the order is the pairs' own.
__global__ void __launch_bounds__(kSlotThreads) place_kernel(SlotsArgs a, int64_t chunk, int chunks) {
  after_previous();
  __shared__ int next[kSlotWarps][TIDE_MAX_EXPERTS];
  __shared__ int part[kSlotWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t from = blockIdx.x * chunk, to = min(a.pairs, from + chunk);
  const int64_t each = chunk / kSlotWarps, w0 = min(to, from + warp * each), w1 = min(to, w0 + each);
  for (int e = threadIdx.x; e < a.experts; e += kSlotThreads)
#pragma unroll
    for (int w = 0; w < kSlotWarps; ++w) next[w][e] = 0;
  __syncthreads();
  for (int64_t i = w0 + lane; i < w1; i += 32) {
    const int e = a.ids[i];
    if ((unsigned)e < (unsigned)a.experts) atomicAdd(&next[warp][e], 1);
  }
  __syncthreads();
  // Experts in turns of a thread each, a running total from turn to turn.
  int base = 0;
  for (int e0 = 0; e0 < a.experts; e0 += kSlotThreads) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e < a.experts) {
      if (chunks == 1) {
        for (int w = 0; w < kSlotWarps; ++w) all += next[w][e];
      } else {
        const int* count = a.counts + e;
#pragma unroll 8
        for (int q = 0; q < chunks; ++q, count += a.experts) {
          const int n = *count;
          all += n;
          before += q < (int)blockIdx.x ? n : 0;
        }
      }
    }
    int sum = all;  // of the experts up to this one
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += v;
    }
    if (lane == 31) part[warp] = sum;
    __syncthreads();
    int turn = 0;
    for (int w = 0; w < kSlotWarps; ++w) {
      if (w < warp) sum += part[w];
      turn += part[w];
    }
    __syncthreads();
    const int start = base + sum - all;
    if (e < a.experts) {
      if (blockIdx.x == 0) a.offsets[e] = start;
      int at = start + before;
      for (int w = 0; w < kSlotWarps; ++w) {
        const int n = next[w][e];
        next[w][e] = at;
        at += n;
      }
    }
    base += turn;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) a.offsets[a.experts] = base;
  __syncthreads();
  for (int64_t i0 = w0; i0 < w1; i0 += 32) {
    const int64_t i = i0 + lane;
    int e = -1;
    if (i < w1) e = a.ids[i];
    if ((unsigned)e >= (unsigned)a.experts) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1));
    int at = 0;
    if (e >= 0) at = next[warp][e];
    __syncwarp();
    if (e >= 0 && rank == 0) next[warp][e] = at + __popc(same);
    __syncwarp();
    if (i < w1) a.slots[i] = e >= 0 ? at + rank : -1;
  }
}

}  // namespace

cudaError_t launch_route(const RouterArgs& a, cudaStream_t stream) {
  return a.bf16 ? run<kForward, uint16_t>(a, stream) : run<kForward, float>(a, stream);
}

cudaError_t launch_route_backward(const RouterArgs& a, cudaStream_t stream) {
  return a.bf16 ? run<kBackward, uint16_t>(a, stream) : run<kBackward, float>(a, stream);
}

int64_t slots_workspace_bytes(int64_t pairs, int64_t experts) {
  const int64_t chunks = ceil_div(pairs, chunk_of(pairs));
  return chunks > 1 ? chunks * experts * 4 : 0;
}

cudaError_t launch_expert_slots(const SlotsArgs& a, cudaStream_t stream) {
  const int64_t chunk = chunk_of(a.pairs);
  const int chunks = (int)ceil_div(a.pairs, chunk);
  if (chunks > 1) {
    const cudaError_t e = launch_early(count_kernel, dim3(chunks), kSlotThreads, 0, 0, stream, a, chunk);
    if (e != cudaSuccess) return e;
  }
  return launch_early(place_kernel, dim3(chunks), kSlotThreads, 0, 0, stream, a, chunk, chunks);
}

}  // namespace tide
