// token_bwd.cuh -- the backward passes of the token path (token_path.cuh).
//
// Prologue, per channel c of a head and token t, with x the projection's
// output, u = conv(x), s = silu(u), y = s r, r = (sum_c s^2 + eps)^-1/2 (q and
// k; y = s for v):
//   ds = r (dy - y (y . dy)),   du = ds sig(u) (1 + u (1 - sig(u)))
//   dx_t = sum_i tap_i du_{t+i}   over the tokens t + i of t's own sequence
//   dtap_i = sum_t du_t x_{t-i}
// u, s and y are recomputed from x, which is read as it was or from its 8-bit
// checkpoint (act_pack.cuh).
//
// Epilogue, per row of dv channels, with n = o r, r = (mean o^2 + eps)^-1/2 and
// out = n weight sig(g):
//   dn = dout weight sig(g),   do = r (dn - n mean(dn n))
//   dg = dout n weight sig(g) (1 - sig(g)),   dweight = sum over rows dout n sig(g)
//
// The sums over tokens (dtap, dweight) go through per-block partial sums and a
// second launch that adds them in a fixed order, so results repeat bit by bit.
#pragma once

#include "act_pack.cuh"
#include "token_path.cuh"

#include <type_traits>

namespace gdn2 {

// PER consecutive values of a row of x: fp32, bf16, or 8-bit codes times the
// row's power of two.
template <typename XT, int PER>
__device__ __forceinline__ void load_act(const XT* p, float power, float (&o)[PER]) {
  if constexpr (sizeof(XT) == 1) {
    static_assert(PER == 2 || PER == 4, "a lane's channels of 64 or 128");
    uint32_t w;
    if constexpr (PER == 2) w = *reinterpret_cast<const uint16_t*>(p);
    else w = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const float2 c = i == 0 ? code_values<0>(w, power) : code_values<2>(w, power);
      o[i] = c.x;
      o[i + 1] = c.y;
    }
  } else {
    Run<XT, PER> r;
    r.load(p);
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = r.v[i];
  }
}

// The hardware's exponential, reciprocal and reciprocal square root on numbers
// that flush to zero below 2^-126: one instruction each, within some 2^-22.  The
// exponential's argument is rounded, so a sigmoid's relative error grows as
// |u| 2^-24 for u < 0 (3e-6 at -50, of a value of 2e-22); where exp(-u) leaves
// fp32's range the sigmoid is 0 or 1.
__device__ __forceinline__ float ex2_ftz(float x) { float y; asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float rcp_ftz(float x) { float y; asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float rsqrt_ftz(float x) { float y; asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); return y; }
__device__ __forceinline__ float2 sigmoid2(float2 u) {
  const float2 e = __fmul2_rn(u, make_float2(-1.44269504f, -1.44269504f));
  const float2 d = __fadd2_rn(make_float2(ex2_ftz(e.x), ex2_ftz(e.y)), make_float2(1.f, 1.f));
  return make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
}
// sig(u) and 1 - sig(u), the latter as exp(-u) sig(u): the difference would lose all
// digits where sig(u) is near 1 (4 % at u = 14).  (Where exp(-u) leaves fp32's
// range sig(u) is 0, and so is their product.)
__device__ __forceinline__ void sigmoids2(float2 u, float2& sg, float2& rest) {
  const float2 t = __fmul2_rn(u, make_float2(-1.44269504f, -1.44269504f));
  const float2 e = make_float2(ex2_ftz(t.x), ex2_ftz(t.y)), d = __fadd2_rn(e, make_float2(1.f, 1.f));
  constexpr float top = 8.5070592e37f;   // 2^126, whose reciprocal is not flushed to zero
  sg = make_float2(rcp_ftz(d.x), rcp_ftz(d.y));
  rest = __fmul2_rn(make_float2(fminf(e.x, top), fminf(e.y, top)), sg);
}

// A launch that adds up what the one before it left may begin while that one
// still runs: next_launch_may_begin in the first, after_last_launch before the
// second reads anything (it returns once the first is complete and visible).
__device__ __forceinline__ void next_launch_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_last_launch() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct TokProBwdArgs {
  const void* x[3];        // projections' outputs [T_total, H, d], or their codes
  const uint8_t* exps[3];  // [T_total, H] with codes
  const float* wt[3];      // taps [H * d, W]
  const float* dy[3];      // gradients of the operator's inputs [T_total, H, d]
  void* dx[3];             // gradients of x
  float* part[3];          // partial tap gradients [grid.x, H * d, W]
  int l2[3];
  const int32_t* cu;
  int N, T, T_total, H;
  int run;                 // consecutive tokens of one warp
};

constexpr int kBwdWarps = 4;
constexpr int kBwdStage = 8;   // tokens per stage of a warp's ring
constexpr int kBwdStages = 2;

// Blocks an SM holds, by registers: the taps, their gradients and the window
// take 16 W + 8 (W + 3) of them at d = 128, wider rows a few more.  At W = 4 bf16
// rows spill with four blocks (164 us against 159 us with three), 8-bit rows do not
// (164 us against 172 us); at W = 3 four are better for both (147 us against 157 us).
// (Measured at d = 128.  The counts are the same at d = 64, whose lanes hold half as much:
// there one block more would fit for bf16 and fp32 rows at W = 4, for all at W = 7 and 8.)
__host__ __device__ constexpr int pro_bwd_blocks(int bytes, int W) {
  return W <= 3 ? (bytes == 4 ? 3 : 4) : W == 4 ? (bytes == 1 ? 4 : 3) : W <= 6 ? 3 : 2;
}

// Dynamic shared memory of the prologue's backward pass: the warps' rings, and
// at the end the warps' tap gradients in the same place.
template <typename XT>
constexpr int pro_bwd_smem(int D, int W) {
  const int ring = kBwdWarps * kBwdStages * kBwdStage * D * ((int)sizeof(XT) + 4), red = kBwdWarps * D * W * 4;
  return ring > red ? ring : red;
}

// The sums over the warp of NV values, NV a power of two: each exchange halves
// the values a lane still carries, so 4 values cost 6 shuffles and 4 to hand
// the sums to every lane, instead of 20.
template <int NV>
__device__ __forceinline__ void warp_sums(float (&v)[NV]) {
  const int lane = threadIdx.x & 31;
  int off = 16;
#pragma unroll
  for (int n = NV; n > 1; n /= 2, off /= 2) {
    const bool up = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < NV / 2; ++j)
      if (j < n / 2) {
        const float give = up ? v[j] : v[j + n / 2], keep = up ? v[j + n / 2] : v[j];
        v[j] = keep + __shfl_xor_sync(0xffffffffu, give, off);
      }
  }
  float s = v[0];
#pragma unroll
  for (; off > 0; off /= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
  // sum j is in the lanes whose upper bits spell j, the first exchange's bit on top
#pragma unroll
  for (int j = 0; j < NV; ++j) v[j] = __shfl_sync(0xffffffffu, s, j * (32 / NV));
}

// grid: (token groups, H, projections).  A warp walks one run of consecutive
// tokens of one head of one projection, two tokens (G) at a time, and W - 1 more on
// either side; a block's warps have neighbouring runs.  Rows arrive through the
// warp's own ring in shared memory (asynchronous copies, no block barrier).  The
// window of x and the gradients that still wait for later tokens stay in
// registers, and so do the tap gradients, over the whole run.
template <typename XT, typename IO, int D, int W>
__global__ void __launch_bounds__(kBwdWarps * 32, pro_bwd_blocks(sizeof(XT), W)) token_prologue_bwd_kernel(const TokProBwdArgs a) {
  constexpr int G = 2;
  static_assert(kBwdStage == 4 * G, "four groups a stage");
  constexpr int PER = D / 32, NP = PER / 2;
  constexpr int ROWX = D * (int)sizeof(XT), ROWG = D * 4, STAGE = kBwdStage * (ROWX + ROWG);
  extern __shared__ __align__(16) uint8_t smem[];
  next_launch_may_begin();
  const int z = blockIdx.z, h = blockIdx.y;
  const XT* __restrict__ x = static_cast<const XT*>(z == 0 ? a.x[0] : z == 1 ? a.x[1] : a.x[2]);
  const uint8_t* __restrict__ exps = z == 0 ? a.exps[0] : z == 1 ? a.exps[1] : a.exps[2];
  const float* __restrict__ dy = z == 0 ? a.dy[0] : z == 1 ? a.dy[1] : a.dy[2];
  IO* __restrict__ dx = static_cast<IO*>(z == 0 ? a.dx[0] : z == 1 ? a.dx[1] : a.dx[2]);
  const bool l2 = (z == 0 ? a.l2[0] : z == 1 ? a.l2[1] : a.l2[2]) != 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = lane * PER;
  float2 tap[W][NP], dtap[W][NP];
  {
    const float* wp = (z == 0 ? a.wt[0] : z == 1 ? a.wt[1] : a.wt[2]) + ((size_t)h * D + c0) * W;
#pragma unroll
    for (int e = 0; e < NP; ++e)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        tap[i][e] = make_float2(wp[2 * e * W + i], wp[(2 * e + 1) * W + i]);
        dtap[i][e] = make_float2(0.f, 0.f);
      }
  }
  const long long ts64 = ((long long)blockIdx.x * kBwdWarps + warp) * a.run;
  if (ts64 < a.T_total) {
    const int ts = (int)ts64, own = min(ts + a.run, a.T_total);
    const int tw = ts - (W - 1);                           // the walk begins with the rows of the first window
    const int end = min(own + W - 1, a.T_total);           // rows from here on are not read
    const int stages = (own + W - 1 - tw + kBwdStage - 1) / kBwdStage;
    uint8_t* ring = smem + warp * (kBwdStages * STAGE);
    // The lane's pieces of 16 bytes in a stage: piece lane % N of rows lane / N,
    // lane / N + 32 / N, ... (N pieces a row).
    constexpr int NX = ROWX / 16, NG = ROWG / 16;
    const size_t rowx = (size_t)a.H * ROWX, rowg = (size_t)a.H * ROWG;   // bytes from a token to the next
    const uint8_t* px = reinterpret_cast<const uint8_t*>(x + (size_t)h * D) + (long long)(tw + lane / NX) * (long long)rowx + lane % NX * 16;
    const uint8_t* pg = reinterpret_cast<const uint8_t*>(dy + (size_t)h * D) + (long long)(tw + lane / NG) * (long long)rowg + lane % NG * 16;
    uint8_t* const ring_end = ring + kBwdStages * STAGE;
    uint8_t* to = ring + lane * 16;                        // where the next stage goes
    int t0 = tw;                                           // its first token
    const auto fetch = [&]() {
      if (t0 >= ts && t0 + kBwdStage <= end) {
#pragma unroll
        for (int r = 0; r < kBwdStage; r += 32 / NX)
          if (32 / NX <= kBwdStage || lane / NX < kBwdStage) cp_async16(to + r * ROWX, px + r * rowx);
#pragma unroll
        for (int r = 0; r < kBwdStage; r += 32 / NG) cp_async16(to + kBwdStage * ROWX + r * ROWG, pg + r * rowg);
      } else {
#pragma unroll
        for (int r = 0; r < kBwdStage; r += 32 / NX) {
          const int t = t0 + r + lane / NX;
          if ((32 / NX <= kBwdStage || lane / NX < kBwdStage) && t >= 0 && t < end) cp_async16(to + r * ROWX, px + r * rowx);
        }
#pragma unroll
        for (int r = 0; r < kBwdStage; r += 32 / NG) {
          const int t = t0 + r + lane / NG;
          if (t >= ts && t < end) cp_async16(to + kBwdStage * ROWX + r * ROWG, pg + r * rowg);
        }
      }
      t0 += kBwdStage;
      px += kBwdStage * rowx;
      pg += kBwdStage * rowg;
      to = to + STAGE < ring_end ? to + STAGE : ring + lane * 16;
    };
    // the powers of 32 rows, one per lane, read 32 rows ahead
    const auto powers = [&](int t) -> float {
      return sizeof(XT) == 1 && t + lane >= 0 && t + lane < end ? pack_power(exps[(size_t)(t + lane) * a.H + h]) : 0.f;
    };
    float pw_now = powers(tw), pw_next = powers(tw + 32);
    // Rows t - (W - 1) .. t + 7 of a stage that begins with token t, and their gradients so far.
    constexpr int X = W - 1 + kBwdStage;
    float2 xw[X][NP], acc[X][NP];
#pragma unroll
    for (int k = 0; k < X; ++k)
#pragma unroll
      for (int e = 0; e < NP; ++e) xw[k][e] = acc[k][e] = make_float2(0.f, 0.f);
    int s0, s1;                                            // the sequence of the token at hand
    seq_bounds(a.cu, a.N, a.T, ts, s0, s1);
#pragma unroll
    for (int k = 0; k < kBwdStages - 1; ++k) {
      if (k < stages) fetch();
      cp_async_commit();
    }
    // Tokens q .. q + G - 1 of the stage that begins with token t.  EDGE: some
    // of the stage's are outside [ts, own), or fewer than W - 1 tokens into their
    // sequence.
    const auto group = [&](auto edge, auto at, int t, const uint8_t* st, IO* pd, int pbase) {
      constexpr bool EDGE = decltype(edge)::value;
      constexpr int q = decltype(at)::value;
      int age[G];                                          // tokens since the sequence's start (EDGE; -1: no token)
      float2 du[G][NP], s[G][NP], k1[G][NP];               // dy, then ds; silu; its derivative
      float sums[2 * G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int tt = t + q + g;
        const bool read = !EDGE || (tt >= 0 && tt < end), live = !EDGE || (tt >= ts && tt < end);
        if (EDGE) {
          if (live && tt >= s1) seq_bounds(a.cu, a.N, a.T, tt, s0, s1);
          age[g] = live ? tt - s0 : -1;
        }
        float r[PER];
        const float p = sizeof(XT) == 1 ? __shfl_sync(0xffffffffu, pw_now, pbase + q + g) : 1.f;
        if (read) load_act<XT, PER>(reinterpret_cast<const XT*>(st + (q + g) * ROWX) + c0, p, r);
        Run<float, PER> dyr;
        if (live) dyr.load(reinterpret_cast<const float*>(st + kBwdStage * ROWX + (q + g) * ROWG) + c0);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          xw[W - 1 + q + g][e] = read ? make_float2(r[2 * e], r[2 * e + 1]) : make_float2(0.f, 0.f);
          du[g][e] = live ? make_float2(dyr.v[2 * e], dyr.v[2 * e + 1]) : make_float2(0.f, 0.f);
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float2 ss = make_float2(0.f, 0.f), sd = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          float2 u = EDGE ? make_float2(0.f, 0.f) : __fmul2_rn(tap[W - 1][e], xw[q + g][e]);
#pragma unroll
          for (int i = EDGE ? W - 1 : W - 2; i >= 0; --i)
            if (!EDGE || i <= age[g]) u = __ffma2_rn(tap[i][e], xw[W - 1 + q + g - i][e], u);
          const float2 sg = sigmoid2(u);
          s[g][e] = __fmul2_rn(u, sg);
          k1[g][e] = __ffma2_rn(s[g][e], __ffma2_rn(sg, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), sg);
          ss = e == 0 ? __fmul2_rn(s[g][e], s[g][e]) : __ffma2_rn(s[g][e], s[g][e], ss);
          sd = e == 0 ? __fmul2_rn(s[g][e], du[g][e]) : __ffma2_rn(s[g][e], du[g][e], sd);
        }
        sums[2 * g] = ss.x + ss.y;
        sums[2 * g + 1] = sd.x + sd.y;
      }
      if (l2) {
        warp_sums<2 * G>(sums);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          // r (dy - y (y . dy)) as r (dy + m s): every factor stays near dy or the row's norm, where
          // r^3 would leave fp32's range from a norm of 1e12 on
          const float r = rsqrt_ftz(sums[2 * g] + kTokEps), m = -(r * sums[2 * g + 1]) * r;
#pragma unroll
          for (int e = 0; e < NP; ++e)
            du[g][e] = __fmul2_rn(make_float2(r, r), __ffma2_rn(make_float2(m, m), s[g][e], du[g][e]));
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const bool mine = !EDGE || (t + q + g >= ts && t + q + g < own);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const float2 d = __fmul2_rn(du[g][e], k1[g][e]);
          constexpr int B = W - 1 + q;                     // row of the group's first token
          // a row's first term starts its sum; the later ones of its window follow token by token
          acc[B + g][e] = !EDGE || age[g] >= 0 ? __fmul2_rn(tap[0][e], d) : make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < W; ++i)
            if (!EDGE || i <= age[g]) {
              if (i > 0) acc[B + g - i][e] = __ffma2_rn(tap[i][e], d, acc[B + g - i][e]);
              if (mine) dtap[i][e] = __ffma2_rn(d, xw[B + g - i][e], dtap[i][e]);
            }
        }
      }
      // rows t + q - (W - 1) .. t + q + G - 1 - (W - 1) are complete
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int tt = t + q + g - (W - 1);
        if (!EDGE || (tt >= ts && tt < own)) {
          Run<IO, PER> o;
#pragma unroll
          for (int e = 0; e < NP; ++e) {
            o.v[2 * e] = acc[q + g][e].x;
            o.v[2 * e + 1] = acc[q + g][e].y;
          }
          o.store(pd + (q + g) * (size_t)a.H * D);
        }
      }
    };
    IO* pd = dx + (long long)(tw - (W - 1)) * (long long)a.H * D + (size_t)h * D + c0;   // row t - (W - 1) of the stage
    const uint8_t* st = ring;
    for (int k = 0; k < stages; ++k) {
      cp_async_wait<kBwdStages - 2>();
      __syncwarp();
      if (k + kBwdStages - 1 < stages) fetch();              // into the place read in step k - 1
      cp_async_commit();
      const int t = tw + k * kBwdStage, pbase = (k * kBwdStage) & 31;   // pbase: the lane with the power of row t
      if (sizeof(XT) == 1 && k > 0 && pbase == 0) {
        pw_now = pw_next;
        pw_next = powers(t + 32);
      }
      // inside: full windows of the sequence at hand, every row that is completed the run's own
      const auto stage = [&](auto edge) {
        group(edge, std::integral_constant<int, 0>{}, t, st, pd, pbase);
        group(edge, std::integral_constant<int, G>{}, t, st, pd, pbase);
        group(edge, std::integral_constant<int, 2 * G>{}, t, st, pd, pbase);
        group(edge, std::integral_constant<int, 3 * G>{}, t, st, pd, pbase);
      };
      if (t - (W - 1) >= ts && t + kBwdStage <= min(own, s1) && t - s0 >= W - 1) stage(std::false_type{});
      else stage(std::true_type{});
#pragma unroll
      for (int r = 0; r < W - 1; ++r)                      // the window moves on
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          xw[r][e] = xw[r + kBwdStage][e];
          acc[r][e] = acc[r + kBwdStage][e];
        }
      pd += kBwdStage * (size_t)a.H * D;
      st = st + STAGE < ring_end ? st + STAGE : ring;
      __syncwarp();                                        // the stage is read: its place may be filled again
    }
  }
  // the block's tap gradients: over its warps through shared memory
  cp_async_wait_all();
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int e = 0; e < NP; ++e)
#pragma unroll
    for (int i = 0; i < W; ++i) {
      red[warp * D * W + (c0 + 2 * e) * W + i] = dtap[i][e].x;
      red[warp * D * W + (c0 + 2 * e + 1) * W + i] = dtap[i][e].y;
    }
  __syncthreads();
  float* part = (z == 0 ? a.part[0] : z == 1 ? a.part[1] : a.part[2]) + ((size_t)blockIdx.x * a.H + h) * D * W;
  for (int j = threadIdx.x; j < D * W; j += kBwdWarps * 32) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kBwdWarps; ++k) sum += red[k * D * W + j];
    part[j] = sum;
  }
}

// y[z][j] = sum_g part[z][g][j], in order
struct SumPartsArgs {
  const float* part[3];
  float* y[3];
  int n[3], groups[3];
};
static __global__ void __launch_bounds__(kTokThreads) sum_parts_kernel(const SumPartsArgs a) {
  after_last_launch();
  const int z = blockIdx.y, j = blockIdx.x * kTokThreads + threadIdx.x;
  const int n = z == 0 ? a.n[0] : z == 1 ? a.n[1] : a.n[2];
  if (j >= n) return;
  const float* p = (z == 0 ? a.part[0] : z == 1 ? a.part[1] : a.part[2]) + j;
  const int groups = z == 0 ? a.groups[0] : z == 1 ? a.groups[1] : a.groups[2];
  float acc = 0.f;
#pragma unroll 8
  for (int g = 0; g < groups; ++g) acc += p[(size_t)g * n];
  (z == 0 ? a.y[0] : z == 1 ? a.y[1] : a.y[2])[j] = acc;
}

struct TokEpiBwdArgs {
  const void *o, *g;
  const uint8_t *o_exps, *g_exps;
  const float* weight;
  const void* dout;
  void *d_o, *d_g;
  float* part;        // [grid, dv]
  long long rows;
};

// kEpiBwdPer values of a row as they lie in memory (16-byte accesses, 8 bytes
// of codes), and as fp32 pairs.
constexpr int kEpiBwdPer = 8;
template <typename T>
struct RawEight {
  static constexpr int BYTES = kEpiBwdPer * (int)sizeof(T), NV = BYTES > 16 ? 2 : 1;
  using V = typename VecT<(BYTES > 16 ? 16 : BYTES)>::T;
  union { V v[NV]; uint32_t w[BYTES / 4]; };
  __device__ __forceinline__ void load(const void* base, size_t at) {
    const V* p = reinterpret_cast<const V*>(static_cast<const T*>(base) + at);
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j] = p[j];
  }
  __device__ __forceinline__ void values(float power, float2 (&o)[kEpiBwdPer / 2]) const {
#pragma unroll
    for (int j = 0; j < kEpiBwdPer / 2; ++j) {
      if constexpr (sizeof(T) == 4) o[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
      else if constexpr (sizeof(T) == 2) o[j] = make_float2(bf16_lo_f(w[j]), bf16_hi_f(w[j]));
      else o[j] = j % 2 == 0 ? code_values<0>(w[j / 2], power) : code_values<2>(w[j / 2], power);
    }
  }
};
template <typename T>
__device__ __forceinline__ void store_eight(void* base, size_t at, const float2 (&o)[kEpiBwdPer / 2]) {
  Run<T, kEpiBwdPer> r;
#pragma unroll
  for (int j = 0; j < kEpiBwdPer / 2; ++j) {
    r.v[2 * j] = o[j].x;
    r.v[2 * j + 1] = o[j].y;
  }
  r.store(static_cast<T*>(base) + at);
}

// DV / 8 lanes per row, 8 channels each; a block walks rows with the grid's
// stride, the next row's loads in flight while it works on one.
template <typename OT, typename GT, typename IO, int DV>
__global__ void __launch_bounds__(kTokThreads, 4) token_epilogue_bwd_kernel(const TokEpiBwdArgs a) {
  constexpr int P = kEpiBwdPer / 2, L = DV / kEpiBwdPer, ROWS = kTokThreads / L;
  __shared__ float red[ROWS][DV];
  next_launch_may_begin();
  const int l = threadIdx.x % L, r = threadIdx.x / L;
  float2 wt[P], dw[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    wt[j] = make_float2(a.weight[l * kEpiBwdPer + 2 * j], a.weight[l * kEpiBwdPer + 2 * j + 1]);
    dw[j] = make_float2(0.f, 0.f);
  }
  RawEight<OT> ro;
  RawEight<GT> rg;
  RawEight<IO> ry;
  float po = 1.f, pg = 1.f;                                  // the powers of codes
  const auto load = [&](long long row) {
    const size_t at = (size_t)row * DV + l * kEpiBwdPer;
    ro.load(a.o, at);
    rg.load(a.g, at);
    ry.load(a.dout, at);
    if (sizeof(OT) == 1) po = pack_power(a.o_exps[row]);
    if (sizeof(GT) == 1) pg = pack_power(a.g_exps[row]);
  };
  const long long stride = (long long)gridDim.x * ROWS;
  long long r0 = (long long)blockIdx.x * ROWS;               // every lane of the block walks the same count of rows
  if (r0 < a.rows) load(r0 + r < a.rows ? r0 + r : r0);
  for (; r0 < a.rows; r0 += stride) {
    const bool live = r0 + r < a.rows;
    float2 o[P], g[P], dy[P];
    ro.values(po, o);
    rg.values(pg, g);
    ry.values(1.f, dy);
    const long long next = r0 + stride;
    if (next < a.rows) load(next + r < a.rows ? next + r : next);
    float2 s2 = make_float2(0.f, 0.f), m2 = s2;
    float2 rest[P];                                          // 1 - sig(g)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      float2 sg;
      sigmoids2(g[j], sg, rest[j]);
      dy[j] = __fmul2_rn(dy[j], sg);                         // dout sig(g)
      g[j] = __fmul2_rn(dy[j], wt[j]);                       // dn
      s2 = __ffma2_rn(o[j], o[j], s2);
      m2 = __ffma2_rn(g[j], o[j], m2);
    }
    float ss = s2.x + s2.y, mm = m2.x + m2.y;
#pragma unroll
    for (int k = L / 2; k > 0; k /= 2) {
      ss += __shfl_xor_sync(0xffffffffu, ss, k);
      mm += __shfl_xor_sync(0xffffffffu, mm, k);
    }
    // n = o rn; mean(dn n) = rn mean(dn o)
    const float rn = rsqrt_ftz(ss * (1.f / DV) + kTokEps), c = -rn * rn * (mm * (1.f / DV));
    const float2 rn2 = make_float2(rn, rn), c2 = make_float2(c, c);
    const size_t at = (size_t)(r0 + r) * DV + l * kEpiBwdPer;
    float2 dg[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const float2 n = __fmul2_rn(o[j], rn2);
      if (live) dw[j] = __ffma2_rn(dy[j], n, dw[j]);
      dg[j] = __fmul2_rn(__fmul2_rn(g[j], n), rest[j]);
      g[j] = __fmul2_rn(rn2, __ffma2_rn(c2, o[j], g[j]));    // do
    }
    if (live) {
      store_eight<IO>(a.d_o, at, g);
      store_eight<IO>(a.d_g, at, dg);
    }
  }
#pragma unroll
  for (int j = 0; j < P; ++j) {
    red[r][l * kEpiBwdPer + 2 * j] = dw[j].x;
    red[r][l * kEpiBwdPer + 2 * j + 1] = dw[j].y;
  }
  __syncthreads();
  if (threadIdx.x < DV) {
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) acc += red[k][threadIdx.x];
    a.part[(size_t)blockIdx.x * DV + threadIdx.x] = acc;
  }
}

// dweight[c] = sum over the blocks' partial sums, in a fixed order: a block has
// 8 channels, 32 threads each with every 32nd partial sum, and then those in order.
constexpr int kSumCols = 8;
static __global__ void __launch_bounds__(256) sum_weight_kernel(const float* __restrict__ part, int groups, int dv, float* y) {
  __shared__ float red[32][kSumCols];
  const int c = blockIdx.x * kSumCols + threadIdx.x % kSumCols, k = threadIdx.x / kSumCols;
  float acc = 0.f;
  after_last_launch();
#pragma unroll 8
  for (int g = k; g < groups; g += 32) acc += part[(size_t)g * dv + c];
  red[k][threadIdx.x % kSumCols] = acc;
  __syncthreads();
  if (k == 0) {
#pragma unroll
    for (int j = 1; j < 32; ++j) acc += red[j][threadIdx.x];
    y[c] = acc;
  }
}

}  // namespace gdn2
