// What follows a block, per token row (shared by moe_combine_norm and the
// tail of moe_layer_forward):
//   g = f / sqrt(mean(f^2) + post_eps) * post_w          (g = f without post_w)
//   h = residual + scale * gate * g                      (out = h rounded once)
//   x_hat = h / sqrt(mean(h^2) + next_eps) * next_w      (from the unrounded h)
//   xq = e4m3(x_hat / s), s = max|x_hat| / 448           (per token or 128 columns)
// f, h, x_hat and the row statistics stay in fp32; every output is rounded
// once, from the fp32 value.
#pragma once

#include "common.cuh"

namespace moe {

// Device-side copy of moe_block_tail plus the output (host: make_tail).
struct TailP {
  const void* residual;
  const bf16* post_w;
  const void* gate;
  const int32_t* gate_row;
  const bf16* next_w;
  bf16* xhat;
  uint8_t* xq;
  float* xscale;
  void* out;
  float post_eps, next_eps, scale;
  int res_f32, out_f32, gate_f32, gate_cols, gate_rows, q_group;
};

// Eight consecutive columns as fp32.
MOE_DEV void load8(const void* p, bool f32, size_t at, float (&v)[8]) {
  if (f32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = s[0], b = s[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8_bf16(*reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + at), v);
  }
}

MOE_DEV void store8_bf16(bf16* p, const float (&v)[8]) {
  uint4 o;
  o.x = pack2_bf16(v[0], v[1]);
  o.y = pack2_bf16(v[2], v[3]);
  o.z = pack2_bf16(v[4], v[5]);
  o.w = pack2_bf16(v[6], v[7]);
  *reinterpret_cast<uint4*>(p) = o;
}

// fp32 columns go out in one 32-byte store where the address allows it (whole
// sectors; two 16-byte stores write every sector in two halves).
MOE_DEV void store8(void* p, bool f32, size_t at, const float (&v)[8]) {
  if (f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + at);
    if (((uintptr_t)d & 31u) == 0) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d),
                   "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                   "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                   "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                   : "memory");
    } else {
      d[0] = make_float4(v[0], v[1], v[2], v[3]);
      d[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
    store8_bf16(static_cast<bf16*>(p) + at, v);
  }
}

// Row of the gate that token t uses, or -1 for an index outside the gate
// (flagged; the row then counts as a zero gate).
MOE_DEV int tail_gate_row(const TailP& p, int t, int* status) {
  if (!p.gate) return 0;
  if (!p.gate_row) return p.gate_rows == 1 ? 0 : t;
  const int r = p.gate_row[t];
  if (r < 0 || r >= p.gate_rows) {
    flag_status(status, MOE_ERR_INVALID_ARG);
    return -1;
  }
  return r;
}

// The token's scalar factor: scale, times the gate when it is one per token.
MOE_DEV float tail_row_factor(const TailP& p, int grow) {
  if (!p.gate || p.gate_cols != 1) return grow < 0 ? 0.f : p.scale;
  if (grow < 0) return 0.f;
  const float g = p.gate_f32 ? static_cast<const float*>(p.gate)[grow]
                             : __bfloat162float(static_cast<const bf16*>(p.gate)[grow]);
  return p.scale * g;
}

// h of eight columns from column c: f the block's output, r its norm factor and
// w its norm weights (unused without post_w), res the residual (zeros without).  A
// row whose gate index is out of range (grow < 0) is the residual alone, whatever f
// holds.
MOE_DEV void tail_h8(const TailP& p, int H, int c, const float (&f)[8], const float (&w)[8], float r,
                     int grow, float factor, const float (&res)[8], float (&h)[8]) {
  float g[8];
  if (p.post_w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = (f[i] * r) * w[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = f[i];
  }
  if (p.gate && p.gate_cols != 1 && grow >= 0) {
    float a[8];
    load8(p.gate, p.gate_f32 != 0, (size_t)grow * H + c, a);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] *= a[i];
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = grow >= 0 ? fmaf(factor, g[i], res[i]) : res[i];
}

// Scale of a row or group whose largest magnitude is m: m / 448, or 1 where that is 0
// (nothing but zeros, or magnitudes whose 448th part is below fp32).
MOE_DEV float tail_scale(float m) {
  const float s = __fdiv_rn(m, 448.0f);
  return s > 0.f ? s : 1.0f;
}

// Both parts of v times s, each rounded by itself.
MOE_DEV float2 mul2(float2 v, float s) {
  float2 d;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mul.rn.f32x2 c, a, b;\n"
      " mov.b64 {%0, %1}, c;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(v.x), "f"(v.y), "f"(s));
  return d;
}

// E4M3 codes of v / s, the IEEE quotient (as moe_quantize_fp8_rows rounds it).  Taken from
// products with 2^-21 less and 2^-21 more than 1 / s, which lie on either side of the
// quotient (three roundings of 2^-24 are between them and it): where both have the same
// code, it is the quotient's.  Only chunks with a value that near to the middle between
// two codes take the divisions (about one chunk in 10^4), and those with a scale so small that
// 1 / s could overflow.  T = 2048, one row per token: H = 4096 17.7 us, 19.7 with divisions
// throughout; H = 8192 28.7, 32.1.
MOE_DEV uint2 tail_e4m3x8(const float (&v)[8], float s) {
  const float inv = __fdiv_rn(1.0f, s), lo = inv * (1.0f - 0x1p-21f), hi = inv * (1.0f + 0x1p-21f);
  uint32_t c[4], apart = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = __nv_cvt_float2_to_fp8x2(mul2(make_float2(v[2 * i], v[2 * i + 1]), lo), __NV_SATFINITE, __NV_E4M3);
    apart |= c[i] ^ __nv_cvt_float2_to_fp8x2(mul2(make_float2(v[2 * i], v[2 * i + 1]), hi), __NV_SATFINITE, __NV_E4M3);
  }
  if (apart != 0 || s < 1e-30f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s)), __NV_SATFINITE,
                                      __NV_E4M3);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

}  // namespace moe
