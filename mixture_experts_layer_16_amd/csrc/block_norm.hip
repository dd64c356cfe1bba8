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
// A row lives in the registers of one team: eight of its elements a lane (sixteen above
// 8,192), so a team is as many wavefronts as the row needs, or 8, 16 or 32 lanes of one.
// Teams walk over rows with the gains in registers and the next row's loads in flight; every
// tensor is read once and written once, and all that crosses lanes are the row sums.  What
// bounds the kernels is memory, and for a few rows the latency of one load, two row sums and
// one store.  Forward, 32,768 rows of 6,144 bf16: 290 us, 5.6 TB/s (the same bytes copied with
// the same hints: 6.0); one row 3.2 us.
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

constexpr int block_threads(int team) { return team <= 64 ? 256 : team; }
constexpr int waves_of(int team) { return team <= 64 ? 1 : team / 64; }

// This thread's team: a scalar where all lanes of a wavefront are of one.
template <int TEAM> __device__ __forceinline__ int own_team() {
  constexpr int kTeams = block_threads(TEAM) / TEAM;
  if constexpr (kTeams == 1) return (int)blockIdx.x;
  const int team = (int)blockIdx.x * kTeams + (int)threadIdx.x / TEAM;
  return TEAM < 64 ? team : __builtin_amdgcn_readfirstlane(team);
}

// Sums of NS values over a team of TEAM threads (a workgroup, where it is more than one
// wavefront; otherwise a wavefront or 8, 16 or 32 lanes of one); every thread ends with the
// same bits.  Two buffers in turn: a wavefront
// writes a buffer again only after the barrier of the sum in between, which all others
// reach after reading it.
template <int TEAM, int NS> struct TeamSum {
  float (*buf)[NS][waves_of(TEAM)];
  int turn = 0;
  __device__ __forceinline__ void operator()(float* v) {
#pragma unroll
    for (int s = 0; s < NS; ++s) v[s] = lanes_total<TEAM < 64 ? TEAM : 64>(v[s]);
    if constexpr (TEAM > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) buf[turn][s][wave] = v[s];
      }
      lds_barrier();
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


// This lane's pieces of a row: piece i is elements (i * TEAM + lane) * 8 .. + 7.
template <int TEAM, int NV> struct Pieces {
  int col[NV];
  bool in[NV];
  __device__ __forceinline__ explicit Pieces(int d) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      col[i] = (i * TEAM + (int)threadIdx.x % TEAM) * 8;
      in[i] = col[i] < d;
    }
  }
  template <bool NT, typename T> __device__ __forceinline__ void load(Row8<T> (&v)[NV], const T* row) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) load_row8<NT>(v[i], row + col[i]);
  }
  __device__ __forceinline__ void gains(float (&v)[NV][8], const float* g) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (in[i]) load8(g + col[i], v[i]);
  }
};

// The gate's values for a group's row.
template <typename T, int TEAM, int NV> struct Gate {
  float a[NV][8];
  __device__ __forceinline__ void at(const Pieces<TEAM, NV>& p, const void* gate, int64_t g, int d, int act) {
    Row8<T> z[NV] = {};
    p.template load<false>(z, static_cast<const T*>(gate) + g * d);
    from(z, act);
  }
  __device__ __forceinline__ void from(const Row8<T> (&z)[NV], int act) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[i][j] = gate_act(z[i].get(j), act);
        __builtin_amdgcn_sched_barrier(0);     // one function at a time: eight side by side are what needs the most registers
      }
    }
  }
};

// NT: rows go past the caches.  COMBINE: y is summed from expert rows.  TOKEN: the gate has a
// row a token (otherwise none, or one for several).
template <typename T, int TEAM, int NV, bool NT, bool COMBINE, bool TOKEN>
__global__ __launch_bounds__(block_threads(TEAM)) void block_norm_kernel(BlockNormArgs a) {
  constexpr int kTeams = block_threads(TEAM) / TEAM;
  __shared__ float buf[2][1][waves_of(TEAM)];
  TeamSum<TEAM, 1> sum{buf};
  const int team = own_team<TEAM>();
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const Pieces<TEAM, NV> p(a.d);
  const float inv_d = 1.f / (float)a.d;
  const T* xs = static_cast<const T*>(a.x);
  const T* ys = static_cast<const T*>(a.y);
  const T* zs = static_cast<const T*>(a.gate);
  Row8<T> x[NV], y[NV], z[NV], x_next[NV], y_next[NV], z_next[NV];
  if (team < a.T) {
    p.template load<NT>(x, xs + (int64_t)team * a.d);
    if (!COMBINE && ys) p.template load<NT>(y, ys + (int64_t)team * a.d);
    if (TOKEN) p.template load<NT>(z, zs + (int64_t)team * a.d);
  }
  float g1[NV][8], g2[NV][8];
  if (a.post_gain) p.gains(g1, a.post_gain);
  if (a.next_gain) p.gains(g2, a.next_gain);
  Gate<T, TEAM, NV> gate;
  int64_t gate_end = 0;                        // of the group whose values these are
  for (int64_t t = team; t < a.T; t += step) {
    const int64_t base = t * a.d;
    if (t + step < a.T) {
      p.template load<NT>(x_next, xs + base + step * a.d);
      if (!COMBINE && ys) p.template load<NT>(y_next, ys + base + step * a.d);
      if (TOKEN) p.template load<NT>(z_next, zs + base + step * a.d);
    }
    float out[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) out[i][j] = p.in[i] ? x[i].get(j) : 0.f;
    if (a.has_y) {
      float v[NV][8];
      if constexpr (COMBINE) {
        const T* yp = static_cast<const T*>(a.y_perm);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
        for (int s0 = 0; s0 < a.k; s0 += 4) {  // four expert rows in flight (eight: the same time)
          Row8<T> e[4][NV];
          float w[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            int row = s0 + s < a.k ? a.slot_row[t * a.k + s0 + s] : -1;
            if (TEAM >= 64) row = __builtin_amdgcn_readfirstlane(row);
            const bool there = (unsigned)row < (unsigned)a.n_rows;
            w[s] = there ? a.topk_w[t * a.k + s0 + s] : 0.f;
            if (there) p.template load<NT>(e[s], yp + (int64_t)row * a.d);
            else
#pragma unroll
              for (int i = 0; i < NV; ++i) e[s][i] = {};
          }
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
              for (int j = 0; j < 8; ++j) v[i][j] = fmaf(w[s], p.in[i] ? e[s][i].get(j) : 0.f, v[i][j]);
        }
        if (a.y_out)
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (p.in[i]) store_row8<NT>(static_cast<T*>(a.y_out) + base + p.col[i], v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = p.in[i] ? y[i].get(j) : 0.f;
      }
      float r = a.branch_scale;
      if (a.post_gain) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
        sum(&ss);
        r *= rsqrtf(ss * inv_d + a.eps);
      }
      if constexpr (TOKEN) gate.from(z, a.gate_act);
      else if (a.gate && t >= gate_end) {
        const uint64_t g = (uint64_t)t / (uint64_t)a.gate_rows, rows = (uint64_t)a.gate_rows;
        gate.at(p, a.gate, (int64_t)g, a.d, a.gate_act);
        gate_end = g + 1 > (uint64_t)a.T / rows ? a.T : (int64_t)((g + 1) * rows);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!p.in[i]) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float n = v[i][j] * r;
          if (a.post_gain) n *= g1[i][j];
          if (a.gate) n *= gate.a[i][j];
          out[i][j] = fmaf(a.res_scale, out[i][j], n);
        }
        store_row8<NT>(static_cast<T*>(a.out) + base + p.col[i], out[i]);
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
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!p.in[i]) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j) out[i][j] *= r * g2[i][j];
        store_row8<NT>(static_cast<T*>(a.h) + base + p.col[i], out[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      x[i] = x_next[i];
      if constexpr (!COMBINE) y[i] = y_next[i];
      if constexpr (TOKEN) z[i] = z_next[i];
    }
  }
}

// Backward.  With o = out, r2 = 1/sqrt(mean(o^2) + eps), r likewise of y, b = bs a g:
//
//   D   = d_out + r2 dh g2 - kap o,  kap = r2^3 sum(dh g2 o) / d
//   dx  = rs D
//   dy  = r (b D - y r m),  m = r sum(b D y) / d
//   d_next_gain = sum_t dh o r2
//   with P = sum of D y r over the rows that share a gate row:
//   d_post_gain = sum of bs a P,  dgate = bs a' g P
//
// sum(b D y) is linear in D, so with c = b y it is sum(c d_out) + r2 sum(c dh g2) - kap
// sum(c o): all six row sums (those three, o^2, y^2, dh g2 o) are taken at once, and neither
// norm's statistics need to be kept by the forward.
//
// A team keeps the column sums of its rows in registers; they go out once at its end (one
// part for the teams of a workgroup), and a second kernel adds the parts in order (no atomics).  Rows are dealt so that a team's
// either cover whole gate groups or lie in one (RowPlan), and the teams' rows next to one
// another where they can: with a run of its own for each team, 16,384 rows of 6,144 bf16
// took 252 us instead of 231 (1.22 GB, 5.3 TB/s; the same bytes copied with the same hints: 6.1).
//
// The gate's and the gain's factors are taken out of the sums over rows: inside, they kept a
// row of each in registers (168 and more a lane at 6,144 columns, 145 now; 12 wavefronts are
// what a CU holds either way, and the time is memory's).  One row ahead is enough: two or
// three took as long.
//
// What is absent is computed with as zeros (a gain or gate as ones): branches inside the
// row cost more registers than the arithmetic costs time.
//
// A value of every team of a workgroup summed into its first team's, the others' zero.
template <int TEAM> __device__ __forceinline__ void join(float (&v)[8], f32x4 (*buf)[TEAM < 64 ? TEAM : 64][2]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int o = TEAM; o < 64; o *= 2)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += __shfl_xor(v[j], o, 64);
  if (lane < TEAM) {
    buf[wave][lane][0] = f32x4{v[0], v[1], v[2], v[3]};
    buf[wave][lane][1] = f32x4{v[4], v[5], v[6], v[7]};
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.f;
    if (threadIdx.x < TEAM)
#pragma unroll
      for (int w = 0; w < 4; ++w) v[j] += buf[w][lane][j / 4][j % 4];
  }
  __syncthreads();
}

template <typename T, int TEAM, int NV, bool NT, bool TOKEN>
__global__ __launch_bounds__(block_threads(TEAM)) void block_norm_backward_kernel(BlockNormBackwardArgs a) {
  constexpr int kTeams = block_threads(TEAM) / TEAM;
  constexpr bool kAhead = TEAM < 1024 && (NV == 1 || sizeof(T) == 2 || !TOKEN);    // the next row fits in registers too
  __shared__ float buf[2][6][waves_of(TEAM)];
  TeamSum<TEAM, 6> sum{buf};
  const int team = own_team<TEAM>();
  const int64_t period = a.gate_rows;
  const bool groups = !TOKEN && a.gate, there = team < a.plan.teams;
  int64_t lo, hi, step = 1, group = 0;
  if (kTeams > 1 && !there) {
    lo = hi = 0;
  } else if (a.plan.teams_per_group > 0) {            // every so many rows of a group
    group = team / a.plan.teams_per_group;
    lo = group * period + team % a.plan.teams_per_group;
    hi = (group + 1) * period;
    step = a.plan.teams_per_group;
  } else if (groups) {                         // whole groups
    lo = (int64_t)team * a.plan.rows;
    hi = lo + a.plan.rows;
    group = (int64_t)((uint64_t)lo / (uint64_t)period);
  } else {
    lo = team;
    hi = a.T;
    step = a.plan.teams;
  }
  if (hi > a.T) hi = a.T;
  const Pieces<TEAM, NV> p(a.d);
  const float inv_d = 1.f / (float)a.d;
  struct Row {
    Row8<T> o[NV], dh[NV], dout[NV], y[NV], z[TOKEN ? NV : 1];
  };
  auto load = [&](Row& q, int64_t t) {
    if (a.next_gain) {
      p.template load<NT>(q.o, static_cast<const T*>(a.out) + t * a.d);
      p.template load<NT>(q.dh, static_cast<const T*>(a.dh) + t * a.d);
    }
    if (a.d_out) p.template load<NT>(q.dout, static_cast<const T*>(a.d_out) + t * a.d);
    if (a.y) p.template load<NT>(q.y, static_cast<const T*>(a.y) + t * a.d);
    if constexpr (TOKEN) p.template load<NT>(q.z, static_cast<const T*>(a.gate) + t * a.d);
  };
  Row q{}, next{};
  if (lo < hi) load(q, lo);

  const bool post = a.post_gain != nullptr, norm_next = a.next_gain != nullptr;
  float g1[NV][8], g2[NV][8], b[NV][8], P[NV][8], acc_post[NV][8], acc_next[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      P[i][j] = acc_post[i][j] = acc_next[i][j] = g2[i][j] = 0.f;
      g1[i][j] = 1.f;
    }
  if (norm_next) p.gains(g2, a.next_gain);
  if (TOKEN && post) p.gains(g1, a.post_gain);
  // the gain and, of its own or of a group's row, the gate
  auto factors = [&](float (&g)[NV][8], Gate<T, TEAM, NV>& gate) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) g[i][j] = gate.a[i][j] = 1.f;
    if (post) p.gains(g, a.post_gain);
    if (a.gate) gate.at(p, a.gate, group, a.d, a.gate_act);
  };
  auto enter = [&]() {
    float g[NV][8];
    Gate<T, TEAM, NV> gate;
    factors(g, gate);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) b[i][j] = a.branch_scale * gate.a[i][j] * g[i][j];
  };
  // the group's rows are through (the team's share of them): to dgate or the team's part of it
  auto leave = [&](float* dgate) {
    float g[NV][8];
    Gate<T, TEAM, NV> gate;
    factors(g, gate);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dg[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = a.branch_scale * P[i][j];
        acc_post[i][j] = fmaf(gate.a[i][j], u, acc_post[i][j]);
        dg[j] = gate_slope(gate.a[i][j], a.gate_act) * (g[i][j] * u);
        P[i][j] = 0.f;
      }
      if (dgate && p.in[i]) store8(dgate + p.col[i], dg);
    }
  };
  if constexpr (!TOKEN) enter();

  for (int64_t t = lo; t < hi; t += step) {
    if (kAhead && t + step < hi) load(next, t + step);
    const int64_t base = t * a.d;
    float slope[TOKEN ? NV : 1][8];
    if constexpr (TOKEN) {
      Gate<T, TEAM, NV> gate;
      gate.from(q.z, a.gate_act);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          b[i][j] = gate.a[i][j];              // times bs g1 below
          slope[i][j] = gate_slope(gate.a[i][j], a.gate_act);
        }
    }
    float s[6] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // o^2, dh g2 o, y^2, c d_out, c dh g2, c o
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ov = q.o[i].get(j), u = q.dh[i].get(j) * g2[i][j], yv = q.y[i].get(j);
        const float cv = (TOKEN ? a.branch_scale * g1[i][j] * b[i][j] : b[i][j]) * yv;
        s[0] = fmaf(ov, ov, s[0]);
        s[1] = fmaf(u, ov, s[1]);
        s[2] = fmaf(yv, yv, s[2]);
        s[3] = fmaf(cv, q.dout[i].get(j), s[3]);
        s[4] = fmaf(cv, u, s[4]);
        s[5] = fmaf(cv, ov, s[5]);
      }
      q.o[i].renew();
      q.dh[i].renew();
      q.dout[i].renew();
      q.y[i].renew();
    }
    sum(s);
    const float r2 = norm_next ? rsqrtf(s[0] * inv_d + a.eps) : 0.f;
    const float kap = norm_next ? r2 * r2 * r2 * (s[1] * inv_d) : 0.f;
    const float r = post ? rsqrtf(s[2] * inv_d + a.eps) : 1.f;
    const float rm = r * r * r * ((s[3] + r2 * s[4] - kap * s[5]) * inv_d);   // r^3 sum(b D y) / d
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float dx[8], dy[8], dz[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ov = q.o[i].get(j), yv = q.y[i].get(j), v = q.dh[i].get(j) * r2;
        const float D = fmaf(-kap, ov, fmaf(v, g2[i][j], q.dout[i].get(j)));
        acc_next[i][j] = fmaf(v, ov, acc_next[i][j]);
        dx[j] = a.res_scale * D;
        const float w = D * (TOKEN ? a.branch_scale * g1[i][j] * b[i][j] : b[i][j]);
        dy[j] = post ? fmaf(r, w, -(rm * yv)) : w;
        if constexpr (TOKEN) {
          const float u = a.branch_scale * D * (yv * r);
          acc_post[i][j] = fmaf(b[i][j], u, acc_post[i][j]);
          dz[j] = slope[i][j] * (g1[i][j] * u);
        } else {
          P[i][j] = fmaf(D, yv * r, P[i][j]);
        }
      }
      if (p.in[i]) {
        store_row8<NT>(static_cast<T*>(a.dx) + base + p.col[i], dx);
        if (a.y) store_row8<NT>(static_cast<T*>(a.dy) + base + p.col[i], dy);
        if (TOKEN) store_row8<NT>(static_cast<T*>(a.dgate) + base + p.col[i], dz);
      }
    }
    if (groups && a.plan.teams_per_group == 0 && (t + 1) % period == 0 && t + 1 < hi) {
      leave(static_cast<float*>(a.dgate) + group * a.d);
      ++group;
      enter();
    }
    if constexpr (kAhead) q = next;
    else if (t + step < hi) load(q, t + step);
  }
  const int64_t at = (int64_t)blockIdx.x * a.d;
  const bool first = kTeams == 1 || threadIdx.x < TEAM;
  if constexpr (kTeams == 1) {
    if constexpr (!TOKEN)
      leave(!groups ? nullptr : a.plan.teams_per_group ? a.part_gate + at : static_cast<float*>(a.dgate) + group * a.d);
  } else {
    __shared__ f32x4 teams[4][TEAM < 64 ? TEAM : 64][2];
    if constexpr (!TOKEN) {
      float* dgate = nullptr;
      if (a.plan.teams_per_group == 0) {
        if (groups && there) dgate = static_cast<float*>(a.dgate) + group * a.d;
      } else if (a.plan.group_parts < a.plan.teams_per_group) {     // the workgroup's teams are of one group
        join<TEAM>(P[0], teams);
        if (first) dgate = a.part_gate + at;
      } else if (there) {
        dgate = a.part_gate + (int64_t)team * a.d;
      }
      leave(dgate);
    }
    if (post) join<TEAM>(acc_post[0], teams);
    if (norm_next) join<TEAM>(acc_next[0], teams);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (!p.in[i] || !first) continue;
    if (post) store8(a.part_post + at + p.col[i], acc_post[i]);
    if (norm_next) store8(a.part_next + at + p.col[i], acc_next[i]);
  }
}

// Column sums of the parts: runs of parts, one for every LANES lanes of four columns each, then
// the runs in order.  blockIdx.y: the post gain, the next gain (those that there are), then the
// gate groups whose rows several workgroups share.  64 columns a workgroup and 64 runs, or 32
// and 128 where that leaves the card with few workgroups of many parts each (launch_reduce).
template <int LANES> __global__ __launch_bounds__(1024) void reduce_parts_kernel(BlockNormBackwardArgs a) {
  constexpr int kRuns = 1024 / LANES;
  __shared__ f32x4 buf[kRuns][LANES];
  int job = blockIdx.y;
  const float* part;
  float* dst;
  int64_t first = 0, count = a.plan.parts;
  if (a.post_gain && job-- == 0) {
    part = a.part_post;
    dst = a.d_post_gain;
  } else if (a.next_gain && job-- == 0) {
    part = a.part_next;
    dst = a.d_next_gain;
  } else {
    part = a.part_gate;
    dst = static_cast<float*>(a.dgate) + (int64_t)job * a.d;
    count = a.plan.group_parts;
    first = (int64_t)job * count;
  }
  const int lane = threadIdx.x % LANES, run = threadIdx.x / LANES, c = ((int)blockIdx.x * LANES + lane) * 4;
  const int64_t per = (count + kRuns - 1) / kRuns;
  const int64_t lo = first + run * per, hi = lo + per < first + count ? lo + per : first + count;
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int64_t w = lo; w < hi; ++w) v += *reinterpret_cast<const f32x4*>(part + w * a.d + c);
  buf[run][lane] = v;
  __syncthreads();
  __shared__ f32x4 eight[8][LANES];
  if (run < 8) {
    v = buf[run * (kRuns / 8)][lane];
#pragma unroll
    for (int q = 1; q < kRuns / 8; ++q) v += buf[run * (kRuns / 8) + q][lane];
    eight[run][lane] = v;
  }
  __syncthreads();
  if (run == 0) {
#pragma unroll
    for (int q = 1; q < 8; ++q) v += eight[q][lane];
    *reinterpret_cast<f32x4*>(dst + c) = v;
  }
}

// The team that holds a row of d elements: eight a lane up to 8,192, then sixteen.  (A whole
// wavefront for rows of 64, seven eighths of it idle: 126,825 rows forward 46.1 us instead of
// 14.1, 200,000 backward 128 instead of 36.  512 threads for rows of 2,496: 19,127 backward
// 148 us, 384 threads 114, forward 80.4 and 79.5; 768 for 4,992: as fast as 640 backward, and
// 109 us against 121 for 16,000 forward.)
template <typename F> void by_width(int64_t d, F f) {
  using std::integral_constant;
  if (d <= 64) f(integral_constant<int, 8>{}, integral_constant<int, 1>{});
  else if (d <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (d <= 256) f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  else if (d <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  else if (d <= 1024) f(integral_constant<int, 128>{}, integral_constant<int, 1>{});
  else if (d <= 1536) f(integral_constant<int, 192>{}, integral_constant<int, 1>{});
  else if (d <= 2048) f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  else if (d <= 384 * 8) f(integral_constant<int, 384>{}, integral_constant<int, 1>{});
  else if (d <= 4096) f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
  else if (d <= 6144) f(integral_constant<int, 768>{}, integral_constant<int, 1>{});
  else if (d <= 8192) f(integral_constant<int, 1024>{}, integral_constant<int, 1>{});
  else f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}

// The backward's: 1,024 threads may have 128 registers each, which it needs more than, so
// up to 8,192 columns 512 threads have sixteen elements each (2,000 rows of 8,192 bf16 47.7 us,
// 75.4 with 1,024 threads; 870 of 7,616 float32 44.3, 83.5).
template <typename F> void by_width_backward(int64_t d, F f) {
  if (d > 6144 && d <= 8192) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  else by_width(d, f);
}

// Rows go past the caches where one tensor of them is larger than what the caches hold of it
// anyway (4 MB of L2 an XCD): 32 MB (32,768 rows of 6,144 bf16 290 us, 311 through them; 2,000
// such rows, 25 MB, 21.0 and 20.5 past them).
bool past_caches(int64_t T, int64_t d, int dtype) { return T * d * (dtype == 1 ? 2 : 4) >= (int64_t(32) << 20); }

template <typename T, int TEAM, int NV, bool NT, bool TOKEN>
void launch_forward(const BlockNormArgs& a, int num_cu, hipStream_t stream) {
  constexpr int threads = block_threads(TEAM), per = threads / TEAM;
  // as many workgroups as a CU's 32 wavefronts hold (16: 352 us for 32,768 rows of 6,144, against 289)
  const int64_t want = (a.T + per - 1) / per, most = (int64_t)num_cu * (32 / (threads / 64));
  const dim3 grid((unsigned)(want < most ? want : most)), block(threads);
  if (a.has_y && a.y == nullptr)
    hipLaunchKernelGGL((block_norm_kernel<T, TEAM, NV, NT, true, TOKEN>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((block_norm_kernel<T, TEAM, NV, NT, false, TOKEN>), grid, block, 0, stream, a);
}

template <typename T, int TEAM, int NV, bool NT, bool TOKEN>
void launch_backward(const BlockNormBackwardArgs& a, hipStream_t stream) {
  constexpr int threads = block_threads(TEAM), per = threads / TEAM;
  const dim3 grid((unsigned)((a.plan.teams + per - 1) / per)), block(threads);
  hipLaunchKernelGGL((block_norm_backward_kernel<T, TEAM, NV, NT, TOKEN>), grid, block, 0, stream, a);
}

// With a launch: the two sums of 511 parts 1,024 wide by 32 columns 14.9 us for the whole call,
// by 64 16.7 (a column a lane and 16 runs: 0.7 more); sums over 2,000 gate groups of 12 parts
// 64 wide 48.8 and 43.3; few parts leave the 128 runs idle.
void launch_reduce(const BlockNormBackwardArgs& a, int64_t jobs, hipStream_t stream) {
  const bool narrow = a.d / 64 * jobs <= 128 && a.plan.parts >= 128;
  const dim3 grid((unsigned)(a.d / (narrow ? 32 : 64)), (unsigned)jobs), block(1024);
  if (narrow) hipLaunchKernelGGL(reduce_parts_kernel<8>, grid, block, 0, stream, a);
  else hipLaunchKernelGGL(reduce_parts_kernel<16>, grid, block, 0, stream, a);
}

// f(nt, token) with both as types
template <typename F> void by_flags(bool nt, bool token, F f) {
  if (nt && token) f(std::true_type{}, std::true_type{});
  else if (nt) f(std::true_type{}, std::false_type{});
  else if (token) f(std::false_type{}, std::true_type{});
  else f(std::false_type{}, std::false_type{});
}

}  // namespace

hipError_t launch_block_norm(int dtype, const BlockNormArgs& a, int num_cu, hipStream_t stream) {
  by_flags(past_caches(a.T, a.d, dtype), a.gate && a.gate_rows == 1, [&](auto nt, auto token) {
    by_width(a.d, [&](auto team, auto nv) {
      constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
      constexpr bool NT = decltype(nt)::value, TOKEN = decltype(token)::value;
      if (dtype == 1) launch_forward<bf16, TEAM, NV, NT, TOKEN>(a, num_cu, stream);
      else launch_forward<float, TEAM, NV, NT, TOKEN>(a, num_cu, stream);
    });
  });
  return hipGetLastError();
}

// Teams of 12 wavefronts a CU on a card of 256 CUs (what their registers allow at once).  Each
// workgroup writes one part of d floats a sum, which the second kernel reads again, so two rows
// a team at least (2,000 rows of 512 bf16: one row 11.0 us, two 9.6) unless that leaves half the
// CUs without work (20 rows of 512: one 6.4, two 7.1), and one workgroup, whose part is the sum,
// where two rows a team are enough for it (8 rows of 512: 4.8, two workgroups 6.4).
RowPlan block_norm_row_plan(int64_t T, int64_t d, int64_t gate_rows) {
  int64_t teams = 0, per = 1;                  // per: teams of a workgroup
  by_width_backward(d, [&](auto team, auto) {
    constexpr int TEAM = decltype(team)::value, waves = waves_of(TEAM);
    per = block_threads(TEAM) / TEAM;
    teams = 256 * (12 / waves > 0 ? 12 / waves : 1) * (TEAM < 64 ? 64 / TEAM : 1);
  });
  int64_t rows = (T + teams - 1) / teams;
  if (T <= 2 * per) rows = (T + per - 1) / per;
  else if (rows < 2 && T > 128 * per) rows = 2;
  RowPlan p{};
  const int64_t groups = gate_rows > 1 ? (T + gate_rows - 1) / gate_rows : 0;
  // a team's longest run of whole groups: narrow rows in many groups of a few rows more than a
  // team's share stay in one team, without a sum over teams for each group
  const int64_t whole = per > 4 && groups >= 1024 ? 4 * rows : rows;
  if (gate_rows <= 1 || gate_rows <= whole) {
    if (gate_rows > 1) rows = (rows + gate_rows - 1) / gate_rows * gate_rows;
    p.rows = rows;
    p.teams = (int)((T + rows - 1) / rows);
  } else {
    const int64_t len = gate_rows < T ? gate_rows : T;     // rows of the longest group
    int64_t of_group = (len + rows - 1) / rows;
    const bool joined = of_group >= per || groups == 1;    // whole workgroups of a group's teams
    if (joined) of_group = (of_group + per - 1) / per * per;
    p.teams_per_group = (int)of_group;
    p.group_parts = (int)(joined ? of_group / per : of_group);
    p.rows = (len + of_group - 1) / of_group;
    p.teams = (int)(groups * of_group);
  }
  p.parts = (int)((p.teams + per - 1) / per);
  return p;
}

hipError_t launch_block_norm_backward(int dtype, const BlockNormBackwardArgs& args, hipStream_t stream) {
  BlockNormBackwardArgs a = args;
  const int64_t groups = a.plan.teams_per_group ? a.plan.teams / a.plan.teams_per_group : 0;
  int64_t jobs = (a.post_gain != nullptr) + (a.next_gain != nullptr) + groups;
  if (a.plan.parts == 1 && (groups == 0 || a.plan.group_parts == 1)) {   // a part is the sum
    a.part_post = a.d_post_gain;
    a.part_next = a.d_next_gain;
    a.part_gate = static_cast<float*>(a.dgate);
    jobs = 0;
  }
  by_flags(past_caches(a.T, a.d, dtype), a.gate && a.gate_rows == 1, [&](auto nt, auto token) {
    by_width_backward(a.d, [&](auto team, auto nv) {
      constexpr int TEAM = decltype(team)::value, NV = decltype(nv)::value;
      constexpr bool NT = decltype(nt)::value, TOKEN = decltype(token)::value;
      if (dtype == 1) launch_backward<bf16, TEAM, NV, NT, TOKEN>(a, stream);
      else launch_backward<float, TEAM, NV, NT, TOKEN>(a, stream);
    });
  });
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (jobs == 0) return hipSuccess;
  launch_reduce(a, jobs, stream);
  return hipGetLastError();
}

}  // namespace moe
