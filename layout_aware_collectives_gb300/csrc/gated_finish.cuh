// Results of the gated block from finished sums, one warp a token: 4 features
// of a block of 128 a lane.
#pragma once

#include "compute_device.cuh"

namespace tide {
namespace {

struct GatedOut {
  int features;
  // h (forward; grad, where it is wanted)
  uint16_t* out;
  int64_t ldo;
  // forward: the 8-bit checkpoint, where it is wanted
  uint8_t *g8, *u8;
  float *gs, *us;
  // grad
  const uint16_t* dh;
  int64_t lddh;
  // bf16, as the tensor cores take them for dX and dW: gradients come out 1.4
  // times as far from their exact values as one bf16 rounding
  uint16_t *dg, *du;
};

// Largest magnitude of a block, as whole numbers, which order alike; NaN is none.
__device__ __forceinline__ float warp_amax(const float4& v) {
  const float m = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, m == m ? __float_as_uint(m) : 0u));
}

// 4 codes a lane, one scale a warp: this lane's part of a token's block.
__device__ __forceinline__ void put_block(float4 v, uint8_t* codes, float* scale, int lane, bool in) {
  float amax = warp_amax(v);
  if (amax == CUDART_INF_F) {
    v = make_float4(no_infinity(v.x), no_infinity(v.y), no_infinity(v.z), no_infinity(v.w));
    amax = warp_amax(v);
  }
  const uint32_t e = scale_exponent(amax);
  const float inv = exponent_inverse(e);
  if (in) *(uint32_t*)codes = pack_e4m3x4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
  if (lane == 0) *scale = exponent_value(e);
}

__device__ __forceinline__ void put_bf16(uint16_t* to, const float4& v) {
  *(uint2*)to = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

template <int ACT>
__device__ __forceinline__ void finish_forward(const GatedOut& o, int64_t token, int block, int lane, const float4& g,
                                               const float4& u) {
  const int col = block * kBlock + lane * 4;
  const bool in = col < o.features;
  if (o.g8) {  // features past the end hold 0
    const int64_t nb = (o.features + kBlock - 1) / kBlock;
    put_block(g, o.g8 + token * o.features + col, o.gs + token * nb + block, lane, in);
    put_block(u, o.u8 + token * o.features + col, o.us + token * nb + block, lane, in);
  }
  if (in)
    put_bf16(o.out + token * o.ldo + col, make_float4(activation<ACT>(g.x) * u.x, activation<ACT>(g.y) * u.y,
                                                      activation<ACT>(g.z) * u.z, activation<ACT>(g.w) * u.w));
}

template <int ACT>
__device__ __forceinline__ void finish_grad(const GatedOut& o, int64_t token, int block, int lane, const float4& gs,
                                            const float4& us) {
  const int col = block * kBlock + lane * 4;
  if (col >= o.features) return;
  const uint2 dh = *(const uint2*)(o.dh + token * o.lddh + col);
  const float d[4] = {bf16_lo(dh.x), bf16_hi(dh.x), bf16_lo(dh.y), bf16_hi(dh.y)};
  const float g[4] = {gs.x, gs.y, gs.z, gs.w}, u[4] = {us.x, us.y, us.z, us.w};
  float dg[4], du[4], h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 s = activation_grad<ACT>(g[i]);
    dg[i] = d[i] * u[i] * s.y, du[i] = d[i] * s.x, h[i] = s.x * u[i];
  }
  const int64_t at = token * o.features + col;
  put_bf16(o.dg + at, make_float4(dg[0], dg[1], dg[2], dg[3]));
  put_bf16(o.du + at, make_float4(du[0], du[1], du[2], du[3]));
  if (o.out) put_bf16(o.out + token * o.ldo + col, make_float4(h[0], h[1], h[2], h[3]));
}

}  // namespace
}  // namespace tide
