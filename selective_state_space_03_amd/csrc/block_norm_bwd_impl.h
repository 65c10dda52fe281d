// The block norm's backward kernel and its launches for one order of gate and norm
// (block_norm_bwd.hip, block_norm_bwd_first.hip: a file each, for the build's time).
#pragma once
#include "block_norm_device.h"

namespace ssm {

struct NormBwdShape {
  int tpr, nch;  // lanes per row, accesses of a lane to a row
  long blocks;
};
template <bool GF>
hipError_t run_norm_bwd(const NormArgs& a, const NormBwdShape& b, hipStream_t s);

namespace {

// Threads of a workgroup: rows of up to 128 lanes share one of 256.
constexpr int norm_block(int tpr) { return tpr < 256 ? 256 : tpr; }

// GF: gate_first.  Parts that are missing cost no branch per element: an absent weight
// is held as ones, an absent gate as z sigmoid = 1.
template <int TPR, int NCH, int XD, int RD, bool GF>
__global__ __launch_bounds__(norm_block(TPR), NCH == 1 ? 3 : TPR * NCH <= 512 ? 2 : 1) void norm_bwd_kernel(NormArgs a) {
  constexpr int BLOCK = norm_block(TPR), TEAMS = BLOCK / TPR;
  __shared__ float sh[32];
  int turn = 0;
  constexpr bool kKnown = XD >= 0;
  const int vec = kKnown ? 8 : a.vec, xd = kKnown ? XD : a.x_dtype, rd = kKnown ? RD : a.res_dtype;
  const int dod = kKnown ? XD : a.dout_dtype, drd = kKnown ? RD : a.dres_dtype;
  const int gd = XD == kF32 ? kF32 : a.grad_dtype;  // (met by the stores alone)
  const int l = threadIdx.x % TPR;
  const long team = static_cast<long>(blockIdx.x) * TEAMS + threadIdx.x / TPR;
  const long teams = static_cast<long>(gridDim.x) * TEAMS;  // a multiple of w_period
  const size_t wo = static_cast<size_t>(team % a.w_period) * a.n;
  const float rn = 1.0f / static_cast<float>(a.n);

  // The weights' columns are the same in every row: in registers with one access per
  // lane, in LDS with two.  Loads among the rows' own would come back after them (loads
  // return in order), which would undo the reading ahead below.
  constexpr bool kRegs = NCH == 1, kLds = !kRegs && NCH == 2;
  __shared__ __align__(16) float wsh[3][kLds ? TPR * NCH * kChunk : 4];
  float wreg[3][8];
  const float* const wsrc[3] = {a.norm_w ? a.norm_w + wo : nullptr, a.scale, a.out_w};
#pragma unroll
  for (int k = 0; k < 3; ++k)
    if (kRegs || kLds) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int i0 = (l + c * TPR) * kChunk;
        if (wsrc[k]) {
          get8(wsrc[k], 0, i0, a.n, kF32, vec, wreg[k]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) wreg[k][i] = 1.0f;
        }
        if (kLds) {
#pragma unroll
          for (int i = 0; i < 8; ++i) wsh[k][i0 + i] = wreg[k][i];  // (read again by this lane only)
        }
      }
    }
  auto weight = [&](int k, int c, float (&v)[8]) {
    const int i0 = (l + c * TPR) * kChunk;
    if (kRegs) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = wreg[k][i];
    } else if (kLds) {
      const float4 x = *reinterpret_cast<const float4*>(&wsh[k][i0]), y = *reinterpret_cast<const float4*>(&wsh[k][i0 + 4]);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else if (wsrc[k]) {
      get8(wsrc[k], 0, i0, a.n, kF32, vec, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    }
  };

  float aw[NCH][8], as[NCH][8], ao[NCH][8];  // this team's column sums
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) aw[c][i] = as[c][i] = ao[c][i] = 0.0f;

  // A row's values as loaded; each is asked for again, for the team's next row, right
  // after its last use, so the loads have the rest of the row before to arrive.
  Raw rx[NCH], rz[NCH], rr[NCH], ro[NCH], re[NCH];
  struct At {
    size_t x, z, dense;
    bool act;
  };
  // every team of a workgroup walks the same number of rows (sums cross the
  // workgroup); a row past the end is computed from row 0 and counts for nothing
  auto at_row = [&](long base) {
    const long row_raw = base + threadIdx.x / TPR;
    At p;
    p.act = row_raw < a.rows;
    const long row = p.act ? row_raw : 0;
    const long call_row = row / a.groups;
    const size_t grp = static_cast<size_t>(row - call_row * a.groups) * a.n;
    p.x = call_row * a.x_stride + grp;
    p.z = call_row * a.z_stride + grp;
    p.dense = static_cast<size_t>(row) * a.n;
    return p;
  };
  auto load_in = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      rx[c] = raw8(a.x, p.x, i0, a.n, xd, vec);
      if (a.z) rz[c] = raw8(a.z, p.z, i0, a.n, xd, vec);
    }
  };
  auto load_out = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      if (a.res && a.out_w) rr[c] = raw8(a.res, p.dense, i0, a.n, rd, vec);
      if (a.dout) ro[c] = raw8(a.dout, p.dense, i0, a.n, dod, vec);
    }
  };
  auto load_res = [&](const At& p) {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      if (a.dres) re[c] = raw8(a.dres, p.dense, (l + c * TPR) * kChunk, a.n, drd, vec);
  };
  const long first = static_cast<long>(blockIdx.x) * TEAMS;
  At cur = at_row(first);
  if (first < a.rows) {
    load_in(cur);
    load_out(cur);
    load_res(cur);
  }
  for (long base = first; base < a.rows; base += teams) {
    const bool act = TEAMS == 1 || cur.act;
    const size_t dense = cur.dense;
    cur = at_row(min(base + teams, a.rows));  // (the row after the last is none: row 0 again)

    // g: the gate z sigmoid(z), h: its derivative sigmoid(z) (1 + z (1 - sigmoid(z)))
    float x[NCH][8], g[NCH][8], h[NCH][8], d[NCH][8];
    float sum[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      widen(rx[c], xd, x[c]);
      if (a.z) {
        float z[8];
        widen(rz[c], xd, z);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float sg = sigmoid(z[i]);
          g[c][i] = z[i] * sg;
          h[c][i] = sg * fmaf(z[i], 1.0f - sg, 1.0f);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[c][i] = 1.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = GF ? x[c][i] * g[c][i] : x[c][i];
        sum[0] = fmaf(y, y, sum[0]);
      }
    }
    load_in(cur);
    float inv = 1.0f;
    if (a.norm_w) {
      row_sums<TPR, 1>(sum, sh, turn);
      inv = 1.0f / sqrtf(sum[0] * rn + a.eps);
    }
    // with an output norm: t and its two sums, then the gradient of t
    if (a.out_w && a.dout) {
      float sum2[2] = {0.0f, 0.0f};
      float t[NCH][8];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float w[8], sc[8], ow[8], dd[8];
        weight(0, c, w);
        weight(1, c, sc);
        weight(2, c, ow);
        if (a.res) {
          widen(rr[c], rd, t[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[c][i] = 0.0f;
        }
        widen(ro[c], dod, dd);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[c][i] = fmaf(x[c][i] * inv * w[i] * g[c][i], sc[i], t[c][i]);
          sum2[0] = fmaf(t[c][i], t[c][i], sum2[0]);
          sum2[1] = fmaf(dd[i] * ow[i], t[c][i], sum2[1]);
        }
      }
      row_sums<TPR, 2>(sum2, sh, turn);
      const float oi = 1.0f / sqrtf(sum2[0] * rn + a.eps);
      const float k = sum2[1] * rn * oi * oi * oi;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float ow[8], dd[8];
        weight(2, c, ow);
        widen(ro[c], dod, dd);
        if (act) {
#pragma unroll
          for (int i = 0; i < 8; ++i) ao[c][i] = fmaf(dd[i] * t[c][i], oi, ao[c][i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = dd[i] * ow[i] * oi;
          // (with one value the difference cancels: what is left is the epsilon's part)
          d[c][i] = TPR == 16 && a.n == 1 ? e * (a.eps * oi * oi) : fmaf(-k, t[c][i], e);
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        if (a.dout) {
          widen(ro[c], dod, d[c]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[c][i] = 0.0f;
        }
      }
    }
    load_out(cur);
    sum[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      if (a.dres) {
        float e[8];
        widen(re[c], drd, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[c][i] += e[i];
      }
      if (act && a.dresidual) put8(a.dresidual, dense, i0, a.n, rd, vec, d[c]);
      float w[8], sc[8];
      weight(0, c, w);
      weight(1, c, sc);
      if (act) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = GF ? x[c][i] * g[c][i] * inv : x[c][i] * inv;  // normalised, before its weight
          as[c][i] = fmaf(d[c][i], GF ? n * w[i] : n * w[i] * g[c][i], as[c][i]);
          aw[c][i] = fmaf(d[c][i] * sc[i], GF ? n : n * g[c][i], aw[c][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[c][i] *= sc[i];
        sum[0] = fmaf(d[c][i] * w[i], x[c][i] * g[c][i] * inv, sum[0]);
      }
    }
    load_res(cur);
    float k = 0.0f;
    if (a.norm_w) {
      row_sums<TPR, 1>(sum, sh, turn);
      k = sum[0] * rn;
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
      float w[8], dz[8];
      weight(0, c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = GF ? x[c][i] * g[c][i] * inv : x[c][i] * inv;
        const float e = GF ? d[c][i] * w[i] : d[c][i] * w[i] * g[c][i];
        // (one value: as above; the epsilon first, as the cube of inv may overflow where it is 0)
        const float dy = TPR == 16 && a.norm_w && a.n == 1 ? a.eps * inv * inv * inv * e : inv * fmaf(-n, k, e);
        dz[i] = (GF ? dy * x[c][i] : d[c][i] * w[i] * n) * h[c][i];
        x[c][i] = GF ? dy * g[c][i] : dy;
      }
      if (act && a.dx) put8(a.dx, dense, i0, a.n, gd, vec, x[c]);
      if (act && a.dz) put8(a.dz, dense, i0, a.n, gd, vec, dz);
    }
  }

  // partial rows: one per workgroup where its teams share a weight row, else one per team
  const size_t cols = a.n;
  if (a.w_period == 1 && TEAMS > 1) {
    constexpr int kRow = TPR * NCH * 8, SLOTS = TPR <= 64 ? 4 : TEAMS;
    __shared__ float acc[SLOTS][kRow];
    const int slot = TPR <= 64 ? threadIdx.x >> 6 : threadIdx.x / TPR;
    for (int which = 0; which < 3; ++which) {
      float (*v)[8] = which == 0 ? aw : which == 1 ? as : ao;
      const bool need = which == 0 ? a.dnorm_w != nullptr : which == 1 ? a.dscale != nullptr : a.dout_w != nullptr;
      if (!need) continue;
#pragma unroll
      for (int c = 0; c < NCH; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float s = v[c][i];
#pragma unroll
          for (int o = TPR; o < 64; o <<= 1) s += __shfl_xor(s, o);
          if ((threadIdx.x & 63) < TPR) acc[slot][(l + c * TPR) * 8 + i] = s;
        }
      __syncthreads();
      for (int i = threadIdx.x; i < a.n; i += BLOCK) {
        float s = acc[0][i];
#pragma unroll
        for (int x = 1; x < SLOTS; ++x) s += acc[x][i];
        a.part[(static_cast<size_t>(blockIdx.x) * 3 + which) * cols + i] = s;
      }
      __syncthreads();
    }
  } else {
    float* p = a.part + static_cast<size_t>(team) * 3 * cols;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int i0 = (l + c * TPR) * kChunk;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < a.n) {
          if (a.dnorm_w) p[i0 + i] = aw[c][i];
          if (a.dscale) p[cols + i0 + i] = as[c][i];
          if (a.dout_w) p[2 * cols + i0 + i] = ao[c][i];
        }
    }
  }
}

template <int TPR, int NCH, bool GF>
hipError_t bwd(const NormArgs& a, long blocks, hipStream_t s) {
  const bool same = (!a.dout || a.dout_dtype == a.x_dtype) && (!a.dres || a.dres_dtype == a.res_dtype) &&
                    (a.x_dtype == kBF16 || a.grad_dtype == kF32);
  const dim3 grid(static_cast<unsigned>(blocks)), block(norm_block(TPR));
  return timed_launch(s, [&] {
    // The types known ahead: 173 instead of 319 us (8192 x 2560, gate, bf16 inputs, f32
    // gradients).  Rows of over 8192 values spill 1.6 kB a lane in every variant: one
    // serves all types.
    if constexpr (TPR * NCH <= 1024) {
      switch (known_types(a, same)) {
        case 0: hipLaunchKernelGGL((norm_bwd_kernel<TPR, NCH, kF32, kF32, GF>), grid, block, 0, s, a); return;
        case 1: hipLaunchKernelGGL((norm_bwd_kernel<TPR, NCH, kBF16, kF32, GF>), grid, block, 0, s, a); return;
        case 2: hipLaunchKernelGGL((norm_bwd_kernel<TPR, NCH, kBF16, kBF16, GF>), grid, block, 0, s, a); return;
        default: break;
      }
    }
    hipLaunchKernelGGL((norm_bwd_kernel<TPR, NCH, -1, -1, GF>), grid, block, 0, s, a);
  });
}

}  // namespace

template <bool GF>
hipError_t run_norm_bwd(const NormArgs& a, const NormBwdShape& b, hipStream_t s) {
  if (b.tpr == 512) return b.nch == 2 ? bwd<512, 2, GF>(a, b.blocks, s) : bwd<512, 4, GF>(a, b.blocks, s);
  if (b.nch == 2) return bwd<256, 2, GF>(a, b.blocks, s);
  switch (b.tpr) {
    case 16: return bwd<16, 1, GF>(a, b.blocks, s);
    case 32: return bwd<32, 1, GF>(a, b.blocks, s);
    case 64: return bwd<64, 1, GF>(a, b.blocks, s);
    case 128: return bwd<128, 1, GF>(a, b.blocks, s);
    default: return bwd<256, 1, GF>(a, b.blocks, s);
  }
}

}  // namespace ssm
