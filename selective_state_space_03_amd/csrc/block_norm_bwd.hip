// Backward of the block norm (formulas in block_norm_fwd.hip) from its inputs: a and
// t are recomputed, so the forward saves nothing.  Three sums per row, each needing
// the one before: sum y^2; sum t^2 with sum dout out_w t; sum dn n (dn the gradient
// of the normalised y, n that value).
//
// Bound by memory: a row's tensors are read once, the next row's while this one is
// computed.  The weights' gradients are column sums: every workgroup keeps running
// sums in registers over the rows it walks and writes one partial row, and a second
// kernel adds the partials in a fixed order (no atomics, the same result every time).
// 8192 x 2560, every part, f32 residual (461 MB): 141 us, 3.3 TB/s, and 6 us for the
// sums; what is left is the three sums in turn at two waves per SIMD (260 us with the
// weights read among the rows' loads, which return in order; 410 us one load at a time).
#include "block_norm_device.h"

namespace ssm {
namespace {

// GF: gate_first.  Parts that are missing cost no branch per element: an absent weight
// is held as ones, an absent gate as z sigmoid = 1.
template <int TPR, int NCH, int XD, int RD, bool GF>
__global__ __launch_bounds__(256, NCH == 1 ? 3 : NCH == 2 ? 2 : 1) void norm_bwd_kernel(NormArgs a) {
  constexpr int TEAMS = 256 / TPR;
  __shared__ float sh[16];
  int turn = 0;
  constexpr bool kKnown = XD >= 0;
  const int vec = kKnown ? 8 : a.vec, xd = kKnown ? XD : a.x_dtype, rd = kKnown ? RD : a.res_dtype;
  const int dod = kKnown ? XD : a.dout_dtype, drd = kKnown ? RD : a.dres_dtype, gd = kKnown ? XD : a.grad_dtype;
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
        // (one value: as above)
        const float dy = TPR == 16 && a.norm_w && a.n == 1 ? inv * inv * inv * a.eps * e : inv * fmaf(-n, k, e);
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
      for (int i = threadIdx.x; i < a.n; i += 256) {
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

// Column sums of the partial rows: 32 columns x 8 runs of partials per workgroup,
// eight loads of a run in flight
__global__ __launch_bounds__(256) void norm_reduce_kernel(NormArgs a) {
  __shared__ float sh[8][33];
  const int which = blockIdx.z, wr = blockIdx.y;
  float* out = which == 0 ? a.dnorm_w : which == 1 ? a.dscale : a.dout_w;
  if (!out) return;
  const int c = threadIdx.x & 31, run = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + c;
  float s = 0.0f;
  if (col < a.n) {
    const float* src = a.part + static_cast<size_t>(which) * a.n + col;
    const int step = 8 * a.w_period;
    for (int p = wr + run * a.w_period; p < a.parts; p += 8 * step) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = p + i * step;
        v[i] = src[static_cast<size_t>(q < a.parts ? q : p) * 3 * a.n];
        if (q >= a.parts) v[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  sh[run][c] = s;
  __syncthreads();
  if (run == 0 && col < a.n) {
    float t = sh[0][c];
#pragma unroll
    for (int i = 1; i < 8; ++i) t += sh[i][c];
    out[static_cast<size_t>(wr) * a.n + col] = t;
  }
}

long gcd(long a, long b) { return b == 0 ? a : gcd(b, a % b); }

struct BwdShape {
  int tpr, nch;
  long blocks;
};

// Lanes per row of the backward kernel, and its workgroups: two per CU (as many
// as its registers allow) where there are rows for them, a whole number of turns round the weight rows.
BwdShape bwd_shape(long rows, int n, int period) {
  BwdShape b;
  const int chunks = (n + kChunk - 1) / kChunk;
  // few registers per lane (three column sums and the row's values are held): two
  // accesses of a lane to a row where 256 lanes allow it
  b.tpr = chunks <= 16 ? 16 : chunks <= 32 ? 32 : chunks <= 64 ? 64 : chunks <= 128 ? 128 : 256;
  b.nch = b.tpr < 256 ? 1 : (chunks + 255) / 256;
  b.nch = b.nch <= 2 ? b.nch : b.nch <= 4 ? 4 : 8;
  const long teams = 256 / b.tpr;
  long blocks = (rows + teams - 1) / teams;
  blocks = blocks < 1 ? 1 : blocks < 512 ? blocks : 512;
  const long unit = period / gcd(period, teams);
  b.blocks = (blocks + unit - 1) / unit * unit;
  return b;
}

template <int TPR, int NCH>
hipError_t bwd(const NormArgs& a, long blocks, hipStream_t s) {
  return timed_launch(s, [&] {
    const dim3 grid(static_cast<unsigned>(blocks));
    auto run = [&](auto after, auto before) {
      if (a.gate_first) hipLaunchKernelGGL(before, grid, dim3(256), 0, s, a);
      else hipLaunchKernelGGL(after, grid, dim3(256), 0, s, a);
    };
    const bool same = (!a.dout || a.dout_dtype == a.x_dtype) && (!a.dres || a.dres_dtype == a.res_dtype) &&
                      a.grad_dtype == a.x_dtype;
    // (rows of more than two accesses per lane spill in every variant: one serves all types)
    switch (NCH <= 2 ? known_types(a, same) : -1) {
      case 0: run(norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kF32, kF32, false>, norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kF32, kF32, true>); break;
      case 1: run(norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kBF16, kF32, false>, norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kBF16, kF32, true>); break;
      case 2: run(norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kBF16, kBF16, false>, norm_bwd_kernel<TPR, (NCH <= 2 ? NCH : 1), kBF16, kBF16, true>); break;
      default: run(norm_bwd_kernel<TPR, NCH, -1, -1, false>, norm_bwd_kernel<TPR, NCH, -1, -1, true>);
    }
  });
}

}  // namespace

int norm_bwd_parts(long rows, int n, int period) {
  const BwdShape b = bwd_shape(rows, n, period);
  return static_cast<int>(period == 1 ? b.blocks : b.blocks * (256 / b.tpr));
}

// (without rows the kernels still run: the weight gradients are then zeros)
hipError_t launch_norm_bwd(const NormArgs& a, hipStream_t s) {
  const BwdShape b = bwd_shape(a.rows, a.n, a.w_period);
  hipError_t e;
  if (b.tpr == 16) e = bwd<16, 1>(a, b.blocks, s);
  else if (b.tpr == 32) e = bwd<32, 1>(a, b.blocks, s);
  else if (b.tpr == 64) e = bwd<64, 1>(a, b.blocks, s);
  else if (b.tpr == 128) e = bwd<128, 1>(a, b.blocks, s);
  else if (b.nch == 1) e = bwd<256, 1>(a, b.blocks, s);
  else if (b.nch == 2) e = bwd<256, 2>(a, b.blocks, s);
  else if (b.nch == 4) e = bwd<256, 4>(a, b.blocks, s);
  else e = bwd<256, 8>(a, b.blocks, s);
  if (e != hipSuccess || (!a.dnorm_w && !a.dscale && !a.dout_w)) return e;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((a.n + 31) / 32, a.w_period, 3), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssm
