// The norms around a block, with its gate and residual scale (forward and backward).
//
//   N(v; g)  = g * v / sqrt(mean(v^2) + eps)
//   n[t]     = N(y[t]; post_gain), or y[t] without a post gain
//   out[t]   = rs * x[t] + bs * a(gate[t / gate_rows]) * n[t]
//   h[t]     = N(out[t]; next_gain)
//
// y[t] is the block's output, or (as moe_combine) the weighted sum of the token's
// expert rows, taken here without a pass of its own through memory.  Without y,
// out = x: the norm before a first block.
//
// A row lives in the registers of one team (a wavefront for d <= 1,024, a workgroup
// above), so every tensor is read once and written once; all that crosses lanes are
// the row sums.  What bounds the kernels is memory, and for a few rows the latency of
// one load, two row sums and one store.
#include "common.h"
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kNone = 0, kSigmoid = 1, kTanh = 2;

// a(z) and, where asked, a'(z)
__device__ __forceinline__ float gate_act(float z, int act) {
  if (act == kSigmoid) return 1.f / (1.f + expf(-z));
  if (act == kTanh) return tanhf(z);
  return z;
}
__device__ __forceinline__ float gate_slope(float a, int act) {
  if (act == kSigmoid) return a * (1.f - a);
  if (act == kTanh) return 1.f - a * a;
  return 1.f;
}

// Sums of NS values over a team of TEAM threads; every thread ends with the same bits.
// Two buffers in turn: a wavefront writes a buffer again only after the barrier of the
// sum in between, which all others reach after reading it.
template <int TEAM, int NS> struct TeamSum {
  float (*buf)[NS][TEAM / 64];
  int turn = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int s = 0; s < NS; ++s) v[s] = wave_sum64(v[s]);
    if constexpr (TEAM > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) buf[turn][s][wave] = v[s];
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        v[s] = buf[turn][s][0];
#pragma unroll
        for (int w = 1; w < TEAM / 64; ++w) v[s] += buf[turn][s][w];
      }
      turn ^= 1;
    }
  }
};

template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void block_norm_kernel(BlockNormArgs a) {
  constexpr int kTeams = TEAM < 256 ? 256 / TEAM : 1;
  __shared__ float buf[2][1][TEAM / 64];
  TeamSum<TEAM, 1> sum{buf};
  const int lane = threadIdx.x % TEAM;
  const int team = __builtin_amdgcn_readfirstlane((int)blockIdx.x * kTeams + (TEAM < 256 ? (int)threadIdx.x / TEAM : 0));
  const int n8 = a.d / 8;
  const float inv_d = 1.f / (float)a.d;
  const T* x = static_cast<const T*>(a.x);
  for (int64_t t = team; t < a.T; t += (int64_t)gridDim.x * kTeams) {
    const int64_t base = t * a.d;
    float out[NV][8], y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + lane;
      if (c < n8) load8(x + base + c * 8, out[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) out[i][j] = 0.f;
    }
    if (a.has_y) {
      if (a.y) {
        const T* yp = static_cast<const T*>(a.y);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = i * TEAM + lane;
          if (c < n8) load8(yp + base + c * 8, y[i]);
          else
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
        }
      } else {
        const T* yp = static_cast<const T*>(a.y_perm);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] = 0.f;
        for (int s = 0; s < a.k; ++s) {
          const int row = __builtin_amdgcn_readfirstlane(a.slot_row[t * a.k + s]);
          if ((unsigned)row >= (unsigned)a.n_rows) continue;
          const float w = a.topk_w[t * a.k + s];
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = i * TEAM + lane;
            if (c >= n8) continue;
            float v[8];
            load8(yp + (int64_t)row * a.d + c * 8, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[i][j] = fmaf(w, v[j], y[i][j]);
          }
        }
        if (a.y_out) {
          T* yo = static_cast<T*>(a.y_out);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int c = i * TEAM + lane;
            if (c < n8) store8(yo + base + c * 8, y[i]);
          }
        }
      }
      float r = 1.f;
      if (a.post_gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(y[i][j], y[i][j], ss);
        sum(&ss);
        r = rsqrtf(ss * inv_d + a.eps);
      }
      r *= a.branch_scale;
      const T* gate = a.gate ? static_cast<const T*>(a.gate) + (t / a.gate_rows) * (int64_t)a.d : nullptr;
      T* o = static_cast<T*>(a.out);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * TEAM + lane;
        if (c >= n8) continue;
        float g[8], z[8];
        if (a.post_gain) load8(a.post_gain + c * 8, g);
        if (gate) load8(gate + c * 8, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float v = y[i][j] * r;
          if (a.post_gain) v *= g[j];
          if (gate) v *= gate_act(z[j], a.gate_act);
          out[i][j] = fmaf(a.res_scale, out[i][j], v);
        }
        store8(o + base + c * 8, out[i]);
      }
    }
    if (a.next_gain) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(out[i][j], out[i][j], ss);
      sum(&ss);
      const float r = rsqrtf(ss * inv_d + a.eps);
      T* h = static_cast<T*>(a.h);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * TEAM + lane;
        if (c >= n8) continue;
        float g[8];
        load8(a.next_gain + c * 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) out[i][j] *= r * g[j];
        store8(h + base + c * 8, out[i]);
      }
    }
  }
}

// Backward.  With o = out, r2 = 1/sqrt(mean(o^2) + eps), r likewise of y:
//
//   D   = d_out + r2 dh g2 - kap o,  kap = r2^3 sum(dh g2 o) / d
//   dx  = rs D
//   dn  = bs a D;  dgate = sum over its rows of bs a' n D
//   dy  = r (dn g - y r m),  m = r sum(dn g y) / d
//   d_post_gain = sum_t dn y r,  d_next_gain = sum_t dh o r2
//
// sum(dn g y) is linear in D, so with c = bs a g y it is sum(c d_out) + r2 sum(c dh g2)
// - kap sum(c o): all six row sums (those three, o^2, y^2, dh g2 o) are taken at once, and
// neither norm's statistics need to be kept by the forward.
//
// A team walks consecutive rows and keeps the column sums in registers; they go out once
// at its end, and a second kernel adds the teams' parts in order (no atomics).  Rows are
// dealt so that a team's rows either cover whole gate groups or lie in one (RowPlan).
template <typename T, int TEAM, int NV>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void block_norm_backward_kernel(BlockNormBackwardArgs a) {
  constexpr int kTeams = TEAM < 256 ? 256 / TEAM : 1;
  __shared__ float buf[2][6][TEAM / 64];
  TeamSum<TEAM, 6> sum{buf};
  const int lane = threadIdx.x % TEAM;
  const int team = __builtin_amdgcn_readfirstlane((int)blockIdx.x * kTeams + (TEAM < 256 ? (int)threadIdx.x / TEAM : 0));
  if (team >= a.plan.teams) return;
  int64_t lo, hi, group_end = 0;
  const int64_t period = a.gate_rows;
  if (a.plan.teams_per_group == 0) {
    lo = (int64_t)team * a.plan.rows;
    hi = lo + a.plan.rows;
  } else {
    const int64_t g = team / a.plan.teams_per_group, j = team % a.plan.teams_per_group;
    lo = g * period + j * a.plan.rows;
    hi = lo + a.plan.rows;
    if (hi > (g + 1) * period) hi = (g + 1) * period;
  }
  if (hi > a.T) hi = a.T;
  const int n8 = a.d / 8;
  const float inv_d = 1.f / (float)a.d;
  const bool sums_gate = a.gate && period > 1;
  float acc_post[NV][8], acc_next[NV][8], acc_gate[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc_post[i][j] = acc_next[i][j] = acc_gate[i][j] = 0.f;

  for (int64_t t = lo; t < hi; ++t) {
    const int64_t base = t * a.d;
    typename Raw16<T>::type o[NV], dh[NV], dout[NV], y[NV], z[NV];
    const int64_t group = a.gate ? t / period : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + lane;
      if (c >= n8) continue;
      if (a.next_gain) {
        o[i] = Raw16<T>::load(static_cast<const T*>(a.out) + base + c * 8);
        dh[i] = Raw16<T>::load(static_cast<const T*>(a.dh) + base + c * 8);
      }
      if (a.d_out) dout[i] = Raw16<T>::load(static_cast<const T*>(a.d_out) + base + c * 8);
      if (a.y) y[i] = Raw16<T>::load(static_cast<const T*>(a.y) + base + c * 8);
      if (a.gate) z[i] = Raw16<T>::load(static_cast<const T*>(a.gate) + group * a.d + c * 8);
    }
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // o^2, dh g2 o, y^2, c d_out, c dh g2, c o
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + lane;
      if (c >= n8) continue;
      float g1[8], g2[8];
      if (a.post_gain) load8(a.post_gain + c * 8, g1);
      if (a.next_gain) load8(a.next_gain + c * 8, g2);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ov = a.next_gain ? Raw16<T>::get(o[i], j) : 0.f;
        const float u = a.next_gain ? Raw16<T>::get(dh[i], j) * g2[j] : 0.f;
        s[0] = fmaf(ov, ov, s[0]);
        s[1] = fmaf(u, ov, s[1]);
        if (a.post_gain) {
          const float yv = Raw16<T>::get(y[i], j);
          float cv = a.branch_scale * g1[j] * yv;
          if (a.gate) cv *= gate_act(Raw16<T>::get(z[i], j), a.gate_act);
          s[2] = fmaf(yv, yv, s[2]);
          if (a.d_out) s[3] = fmaf(cv, Raw16<T>::get(dout[i], j), s[3]);
          s[4] = fmaf(cv, u, s[4]);
          s[5] = fmaf(cv, ov, s[5]);
        }
      }
    }
    sum(s);
    const float r2 = rsqrtf(s[0] * inv_d + a.eps);
    const float kap = a.next_gain ? r2 * r2 * r2 * (s[1] * inv_d) : 0.f;
    const float r = a.post_gain ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float m = r * r * ((s[3] + r2 * s[4] - kap * s[5]) * inv_d);   // r^2 sum(dn g y) / d
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * TEAM + lane;
      if (c >= n8) continue;
      float g1[8], g2[8], dx[8], dy[8], dz[8];
      if (a.post_gain) load8(a.post_gain + c * 8, g1);
      if (a.next_gain) load8(a.next_gain + c * 8, g2);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float D = a.d_out ? Raw16<T>::get(dout[i], j) : 0.f;
        if (a.next_gain) {
          const float ov = Raw16<T>::get(o[i], j), dhv = Raw16<T>::get(dh[i], j);
          D += r2 * (dhv * g2[j]) - kap * ov;
          acc_next[i][j] = fmaf(dhv, ov * r2, acc_next[i][j]);
        }
        dx[j] = a.res_scale * D;
        if (a.y) {
          const float yr = Raw16<T>::get(y[i], j) * r;
          float dn = a.branch_scale * D;
          if (a.gate) {
            const float av = gate_act(Raw16<T>::get(z[i], j), a.gate_act);
            dz[j] = dn * gate_slope(av, a.gate_act) * (a.post_gain ? yr * g1[j] : yr);
            if (sums_gate) acc_gate[i][j] += dz[j];
            dn *= av;
          }
          if (a.post_gain) {
            acc_post[i][j] = fmaf(dn, yr, acc_post[i][j]);
            dy[j] = r * (dn * g1[j]) - m * yr;
          } else {
            dy[j] = dn;
          }
        }
      }
      store8(static_cast<T*>(a.dx) + base + c * 8, dx);
      if (a.y) store8(static_cast<T*>(a.dy) + base + c * 8, dy);
      if (a.gate && !sums_gate) store8(static_cast<T*>(a.dgate) + base + c * 8, dz);
    }
    if (sums_gate && a.plan.teams_per_group == 0 && (t + 1 == hi || (t + 1) % period == 0)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = i * TEAM + lane;
        if (c < n8) store8(static_cast<float*>(a.dgate) + group * a.d + c * 8, acc_gate[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc_gate[i][j] = 0.f;
      }
    }
  }
  const int64_t at = (int64_t)team * a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = i * TEAM + lane;
    if (c >= n8) continue;
    if (a.post_gain) store8(a.part_post + at + c * 8, acc_post[i]);
    if (a.next_gain) store8(a.part_next + at + c * 8, acc_next[i]);
    if (a.plan.teams_per_group) store8(a.part_gate + at + c * 8, acc_gate[i]);
  }
}

// Column sums of the teams' parts, 64 columns a workgroup, four runs of teams added in
// order.  blockIdx.y: the post gain, the next gain (those that there are), then the gate
// groups whose rows several teams share.
__global__ __launch_bounds__(256) void reduce_parts_kernel(BlockNormBackwardArgs a) {
  __shared__ float buf[4][64];
  int job = blockIdx.y;
  const float* part;
  float* dst;
  int64_t first = 0, count = a.plan.teams;
  if (a.post_gain && job-- == 0) {
    part = a.part_post;
    dst = a.d_post_gain;
  } else if (a.next_gain && job-- == 0) {
    part = a.part_next;
    dst = a.d_next_gain;
  } else {
    part = a.part_gate;
    dst = static_cast<float*>(a.dgate) + (int64_t)job * a.d;
    count = a.plan.teams_per_group;
    first = (int64_t)job * count;
  }
  const int c = (int)blockIdx.x * 64 + (threadIdx.x & 63), run = threadIdx.x >> 6;
  const int64_t per = (count + 3) / 4;
  const int64_t lo = first + run * per, hi = lo + per < first + count ? lo + per : first + count;
  float v = 0.f;
#pragma unroll 8
  for (int64_t w = lo; w < hi; ++w) v += part[w * a.d + c];
  buf[run][threadIdx.x & 63] = v;
  __syncthreads();
  if (run == 0) dst[c] = (buf[0][threadIdx.x] + buf[1][threadIdx.x]) + (buf[2][threadIdx.x] + buf[3][threadIdx.x]);
}

// The team that holds a row of d elements: the fewest threads that hold it in at most
// four pieces of eight elements each, a whole workgroup above 1,024.
template <typename F> void by_width(int64_t d, F f) {
  if (d <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (d <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (d <= 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (d <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (d <= 6144) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 3>{});
  else if (d <= 8192) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

}  // namespace

hipError_t launch_block_norm(int dtype, const BlockNormArgs& a, int num_cu, hipStream_t stream) {
  by_width(a.d, [&](auto team, auto nv) {
    constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
    const int per = TEAM < 256 ? 256 / TEAM : 1;
    const int64_t want = (a.T + per - 1) / per, most = (int64_t)num_cu * 16;
    const dim3 grid((unsigned)(want < most ? want : most)), block(TEAM < 256 ? 256 : TEAM);
    if (dtype == 1) hipLaunchKernelGGL((block_norm_kernel<bf16, TEAM, NV>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((block_norm_kernel<float, TEAM, NV>), grid, block, 0, stream, a);
  });
  return hipGetLastError();
}

RowPlan block_norm_row_plan(int64_t T, int64_t d, int64_t gate_rows) {
  // at most 512 workgroups' worth of teams: each team writes one part of d floats a sum
  const int64_t teams = d <= 1024 ? 2048 : 512;
  int64_t rows = (T + teams - 1) / teams;
  RowPlan p{};
  if (gate_rows <= 1 || gate_rows <= rows) {
    if (gate_rows > 1) rows = (rows + gate_rows - 1) / gate_rows * gate_rows;
    p.rows = rows;
    p.teams = (int)((T + rows - 1) / rows);
  } else {
    const int64_t groups = (T + gate_rows - 1) / gate_rows;
    const int64_t len = gate_rows < T ? gate_rows : T;     // rows of the longest group
    p.teams_per_group = (int)((len + rows - 1) / rows);
    p.rows = (len + p.teams_per_group - 1) / p.teams_per_group;
    p.teams = (int)(groups * p.teams_per_group);
  }
  return p;
}

hipError_t launch_block_norm_backward(int dtype, const BlockNormBackwardArgs& a, hipStream_t stream) {
  by_width(a.d, [&](auto team, auto nv) {
    constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
    const int per = TEAM < 256 ? 256 / TEAM : 1;
    const dim3 grid((unsigned)((a.plan.teams + per - 1) / per)), block(TEAM < 256 ? 256 : TEAM);
    if (dtype == 1) hipLaunchKernelGGL((block_norm_backward_kernel<bf16, TEAM, NV>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((block_norm_backward_kernel<float, TEAM, NV>), grid, block, 0, stream, a);
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t groups = a.plan.teams_per_group ? a.plan.teams / a.plan.teams_per_group : 0;
  const int64_t jobs = (a.post_gain != nullptr) + (a.next_gain != nullptr) + groups;
  if (jobs == 0) return hipSuccess;
  hipLaunchKernelGGL(reduce_parts_kernel, dim3((unsigned)(a.d / 64), (unsigned)jobs), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe
