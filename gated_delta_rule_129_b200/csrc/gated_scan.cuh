// gated_scan.cuh -- the gated linear recurrence
//
//   h_t = alpha_t h_{t-1} + w_t v_t,   alpha_t = exp(log_alpha_t),   out_t = h_t
//
// channel by channel: the operator's state with one key channel, k = q = 1, no
// erase and scale 1.  Its backward pass, with g_t the gradient reaching h_t and
// r_t = alpha_t g_t what flows on to h_{t-1}:
//
//   g_t = dO_t + r_{t+1}          (r_{T+1} = dhT)
//   dv_t = w_t g_t,  dw_t = v_t g_t,  dlog_alpha_t = alpha_t h_{t-1} g_t,  dh0 = r_1
//
// Both directions are bound by HBM traffic (12 and 24 bytes a value in bf16), so
// each is one pass over the data.  A cluster of CL blocks walks one sequence's
// chunks of 64 tokens for a slab of 64 channels, CL chunks a step (forward, or
// from the end); the next step's rows come into shared memory by asynchronous
// copies meanwhile.  Warp k of a block has tokens 8k .. 8k + 7 of the block's
// chunk in registers, a lane two neighbouring channels.
//
// Over any run of tokens the recurrence is the affine map x -> A x + H with A
// the product of the decays.  A chunk's map is folded from its warps' maps and
// written to every block of the cluster through distributed shared memory; each
// block then folds the maps of the step, in sequence order, onto the state that
// entered the step.  Only this fold, CL fused multiply-adds, depends on the step
// before.  Maps are always folded onto a state chunk by chunk, never composed
// with one another, so neither CL nor the packing changes a bit of the results.
//
// Measured, 16 heads of 128, bf16: forward 16K x 1 (CL = 8) 72 us, 2K x 8 (CL = 1)
// 66 us, 85 % and 92 % of the measured copy bandwidth; backward 140 and 147 us,
// 87 % and 84 %; 32 packed sequences of 256 to 8192 tokens 100 % and 94 %: once
// blocks come and go on their own, waits no longer coincide.  A single pass that looked back over published tiles instead of walking
// took 202 us forward (160 KB of registers an SM in flight over 14 us waits); one
// thread per channel 9.3 ms.  With few channels a step's length bounds it: 16K x 1
// with 256 channels 46 to 54 us (by the GPU), 32 steps of 1.4 to 1.7 us.
#pragma once

#include "common.cuh"
#include "tc.cuh"

namespace gdn2 {

constexpr int kScanTok = 8;                        // tokens per warp
constexpr int kScanWarps = kChunk / kScanTok;
constexpr int kScanThr = kScanWarps * 32;
constexpr int kScanSlab = 64;                      // channels of a block: two per lane
constexpr int kScanMaxCluster = 8;

struct ScanArgs {
  const void *v, *dO;
  const float *la, *w, *h0, *dhT;
  void* out;
  float *hT, *states;           // states: [chunks, D] at chunk starts, or nullptr
  float *dv, *dla, *dw, *dh0;
  SeqMap map;                   // chunk_off is nullptr for dense rows, and for few packed sequences
  const int32_t* order;         // with chunk_off: the sequences, longest first; nullptr: as they are numbered
  int longest_first;            // without: whether blocks begin with the longest
  int T_total, seqlens_code;    // without: what cu_seqlens ends with; the status if it does not
  int D, slabs;                 // channels of a token (a multiple of 64); D / 64
  int* status;                  // set by the launch itself, or by the plan that wrote chunk_off
  int timeout_code;             // stored there by a wait that gave up
  unsigned long long wait_ns;   // after which a wait for a step's maps gives up
};

__device__ __forceinline__ void store_io2(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store_io2(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ float2 load_io2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 load_io2(const __nv_bfloat16* p) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
  return make_float2(bf16_lo_f(u), bf16_hi_f(u));
}
// A x + H on two channels, packed arithmetic (each half rounds like fmaf).
__device__ __forceinline__ float2 apply_map(float4 m, float2 x) {
  return __ffma2_rn(make_float2(m.x, m.y), x, make_float2(m.z, m.w));
}

// exp of a log-decay.  Slow decays, |x| < 2^-6, reach over hundreds of tokens
// and their errors add up along the way: those take the series to x^3 (the next
// term is under 2^-28), whose last sum rounds to half an ulp.  Others take the
// hardware's 2^t, t = x log2 e rounded, relative error under 2^-22.4, times
// 1 + r with r = x - t ln 2 (ln 2 in two parts, as Cody and Waite reduce
// arguments), so that steep decays keep that error too.  Arguments under -104
// count as -104, whose exponential is 0; NaN stays NaN.  (Packed arithmetic gained
// nothing here: its constants want register pairs.)
__device__ __forceinline__ float decay(float x) {
  constexpr float L = 1.44269504f, HI = -0.693147182f, LO = 1.90465421e-9f;   // HI + LO = -ln 2
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(-104.f));
  const float t = x * L, r = fmaf(t, LO, fmaf(t, HI, x));
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
  y = fmaf(y, r, y);
  const float p = fmaf(fmaf(fmaf(x, 1.f / 6, 0.5f), x, 1.f), x, 1.f);
  return fabsf(x) < 0.015625f ? p : y;
}
__device__ __forceinline__ float2 decay2(float2 x) { return make_float2(decay(x.x), decay(x.y)); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of a shared-memory variable in the cluster's block `rank`.
__device__ __forceinline__ uint32_t cluster_address(const void* own, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(own)), "r"(rank));
  return at;
}
// 16 bytes to the same variable of block `rank`; their arrival counts on that
// block's barrier `bar`.  (A cluster barrier instead, whose release waits for the
// block's stores to global memory too, cost the backward pass 5 %.)
__device__ __forceinline__ void store_cluster_async(void* own, uint64_t* bar, uint32_t rank, float4 v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
               ::"r"(cluster_address(own, rank)), "r"(__float_as_uint(v.x)), "r"(__float_as_uint(v.y)),
                 "r"(__float_as_uint(v.z)), "r"(__float_as_uint(v.w)), "r"(cluster_address(bar, rank)) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"((uint32_t)__cvta_generic_to_shared(bar)), "r"(parity) : "memory");
  return ok != 0;
}
// The rest of a thread's wait for a step's maps, at most a.wait_ns; false: it gave up
// and the status word says so.  A thread that gave up waits no more (a single try
// takes 4 us at most), sends no maps and arms no barrier, so one is armed only by a
// thread that saw its phase before complete.  The cluster's other blocks then miss
// this one's maps and give up too, their waits having begun about when this one's
// did: a cluster takes about one limit longer than its walk, however many steps
// that has, and leaves the outputs unspecified.
__device__ __forceinline__ bool wait_longer(uint64_t* bar, uint32_t parity, const ScanArgs& a) {
  const uint64_t t0 = tc::global_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if ((it & 15u) == 0 && tc::global_ns() - t0 > a.wait_ns) break;
  }
  atomicExch(a.status, a.timeout_code);
  return false;
}
// The end of a cluster's walk: no block ends while others may still write to it.
// Maps on their way to a block that gave up are not waited for: they get ample time
// to land.
__device__ __forceinline__ void end_cluster_walk(bool lost) {
  cluster_sync();
  if (!lost) return;
  const uint64_t t0 = tc::global_ns();
  while (tc::global_ns() - t0 < 100000ull) {}
}

// What a block walks: one sequence, one slab.
struct ScanSeq {
  int n, slab, t0, len, chunks, chunk0;   // sequence, slab, first token, tokens, chunks, index of the first
};

// Few packed sequences: every block checks cu_seqlens and numbers the chunks by
// itself, one thread a sequence, which saves the launch that does so for many
// (9 sequences, 5.8K tokens: 20 -> 17 us a call).  `place` counts the sequences from
// the longest if a.longest_first.  A malformed array gives a sequence without chunks.
constexpr int kScanLocal = 64;
__device__ __forceinline__ ScanSeq scan_seq_local(const ScanArgs& a, int place) {
  __shared__ int s_chunks[kScanLocal], s_n;
  ScanSeq q;
  const int N = a.map.N, i = threadIdx.x, lane = i & 31;
  bool bad = false;
  int mine = 0;
  if (i < N) {
    const int b = a.map.cu[i], e = a.map.cu[i + 1];
    bad = e < b || (i == 0 && b != 0) || (i == N - 1 && e != a.T_total);
    s_chunks[i] = mine = bad ? 0 : (e - b + kChunk - 1) / kChunk;
  }
  if (i == 0) s_n = place;
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && i == 0) *a.status = bad ? a.seqlens_code : 0;
  q.n = place;
  if (a.longest_first && !bad) {
    if (i < N) {
      int before = 0;
      for (int m = 0; m < N; ++m) before += s_chunks[m] > mine || (s_chunks[m] == mine && m < i);
      if (before == place) s_n = i;
    }
    __syncthreads();
    q.n = s_n;
  }
  int sum = 0;
  for (int m = lane; m < q.n; m += 32) sum += s_chunks[m];
  q.chunk0 = __reduce_add_sync(0xffffffffu, sum);
  q.chunks = bad ? 0 : s_chunks[q.n];
  return q;
}

__device__ __forceinline__ ScanSeq scan_seq(const ScanArgs& a, int cl) {
  ScanSeq q;
  const int pair = blockIdx.x / cl, place = pair / a.slabs;
  if (a.map.cu && !a.map.chunk_off) {
    q = scan_seq_local(a, place);
  } else if (a.map.cu) {
    // a malformed cu_seqlens left no chunks at all: nothing below is then touched
    q.n = a.order ? a.order[place] : place;
    q.chunk0 = a.map.chunk_off[q.n];
    q.chunks = a.map.chunk_off[q.n + 1] - q.chunk0;
  } else {
    q.n = place;
    q.chunks = (a.map.T + kChunk - 1) / kChunk;
    q.chunk0 = q.n * q.chunks;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  }
  q.slab = pair - place * a.slabs;
  q.t0 = a.map.seq_begin(q.n);
  q.len = q.chunks > 0 ? a.map.seq_end(q.n) - q.t0 : 0;
  return q;
}

// The rows of chunk j for the block's slab into shared memory, 16 bytes a copy
// (rows past the sequence's end stay as they were: they are never used).  The
// address is formed anew each time: registers are what the walks are short of.
template <typename T>
__device__ __forceinline__ void fetch_rows(T (*dst)[kScanSlab], const T* src, const ScanArgs& a, const ScanSeq& q, int j) {
  constexpr int PIECES = kScanSlab * (int)sizeof(T) / 16, STEP = kScanThr / PIECES;
  const int r0 = threadIdx.x / PIECES, rows = q.len - j * kChunk;
  char* to = reinterpret_cast<char*>(dst) + threadIdx.x * 16;
  const T* from = src + (size_t)(q.t0 + j * kChunk + r0) * a.D + q.slab * kScanSlab + threadIdx.x % PIECES * (16 / (int)sizeof(T));
#pragma unroll
  for (int r = 0; r < kChunk; r += STEP)
    if (rows >= kChunk || r0 + r < rows) cp_async16(to + r * PIECES * 16, from + (size_t)r * a.D);
}

// Stages lie on 128-byte lines of shared memory: on a 16-byte offset from them the
// copies' 32-byte sectors straddle lines, and the forward pass took 95 us instead of
// 72 us (16K x 1).
template <typename IO>
struct ScanStageFwd {
  float la[kChunk][kScanSlab], w[kChunk][kScanSlab];
  IO v[kChunk][kScanSlab];
};
template <typename IO>
struct ScanStageBwd {
  float la[kChunk][kScanSlab], w[kChunk][kScanSlab];
  IO v[kChunk][kScanSlab], dO[kChunk][kScanSlab];
};

// Forward: step s's loads and maps come before step s - 1's states and outputs,
// so a chunk's map has a whole step to reach the other blocks.
// (fp32 rows leave two blocks an SM room for the maps of four ranks.)
template <typename IO>
constexpr int scan_max_cluster() { return sizeof(IO) == 4 ? kScanMaxCluster / 2 : kScanMaxCluster; }
template <typename IO>
struct ScanFwdMaps {
  float4 warp[2][kScanWarps][32];                  // by the step's parity
  float4 chunk[4][scan_max_cluster<IO>()][32];     // by the step's number modulo 4, and the rank
  uint64_t arrived[4];                             // the step's maps are here
};

template <typename IO, bool CLUSTER>
__global__ void __launch_bounds__(kScanThr, 2) gated_scan_fwd_kernel(const ScanArgs a, int cluster) {
  const int cl = CLUSTER ? cluster : 1;
  constexpr int R = kScanTok, NW = kScanWarps;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Stage = ScanStageFwd<IO>;
  Stage* stages = reinterpret_cast<Stage*>(smem_raw);
  __shared__ __align__(128) ScanFwdMaps<IO> maps;
  bool lost = false;                                     // a wait of this thread gave up
  const ScanSeq q = scan_seq(a, cl);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = CLUSTER ? (int)cluster_rank() : 0;
  const int ch = q.slab * kScanSlab + 2 * lane;
  const size_t sidx = (size_t)q.n * a.D + ch;
  float2 x = make_float2(0.f, 0.f);                      // the state that enters the step
  if (a.h0) x = load_io2(a.h0 + sidx);
  if (q.len == 0) {
    if (a.hT && rank == 0 && warp == 0) store_io2(a.hT + sidx, x.x, x.y);
    return;
  }
  const int steps = (q.chunks + cl - 1) / cl;
  const auto fetch = [&](int s) {
    const int j = s * cl + rank;
    if (s < steps && j < q.chunks) {
      Stage& st = stages[s & 1];
      fetch_rows(st.la, a.la, a, q, j);
      fetch_rows(st.w, a.w, a, q, j);
      fetch_rows(st.v, static_cast<const IO*>(a.v), a, q, j);
    }
    cp_async_commit();
  };
  fetch(0);
  fetch(1);
  if (CLUSTER) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < 4; ++i) tc::mbar_init(&maps.arrived[i], 1);
      tc::fence_mbar_init();
    }
    cluster_sync();                                      // every block runs, its barriers ready, before any writes to it
  }
  const auto tokens = [&](int s) { return min(R, min(kChunk, q.len - (s * cl + rank) * kChunk) - warp * R); };
  // decays and inputs of the warp's tokens in a step, and its map
  const auto load = [&](int s, float2 (&al)[R], float2 (&u)[R]) {
    const Stage& st = stages[s & 1];
    const int n = tokens(s);
    float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f);
    const auto token = [&](int i) {
      const int r = warp * R + i;
      al[i] = decay2(load_io2(&st.la[r][2 * lane]));
      u[i] = __fmul2_rn(load_io2(&st.w[r][2 * lane]), load_io2(&st.v[r][2 * lane]));
      A = __fmul2_rn(A, al[i]);
      H = __ffma2_rn(al[i], H, u[i]);
    };
    if (n >= R) {
#pragma unroll
      for (int i = 0; i < R; ++i) token(i);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) token(i);
    }
    maps.warp[s & 1][warp][lane] = make_float4(A.x, A.y, H.x, H.y);
  };
  // the chunk's map, from its warps' maps, to every block of the cluster
  const auto hand_out = [&](int s) {
    if (CLUSTER && lost) return;
    if (CLUSTER && lane == 0) tc::mbar_arrive_expect_tx(&maps.arrived[s & 3], min(cl, q.chunks - s * cl) * 512u);
    if (s * cl + rank >= q.chunks) return;
    const float4 m0 = maps.warp[s & 1][0][lane];
    float2 A = make_float2(m0.x, m0.y), H = make_float2(m0.z, m0.w);
#pragma unroll
    for (int k = 1; k < NW; ++k) {
      const float4 mk = maps.warp[s & 1][k][lane];
      H = apply_map(mk, H);
      A = __fmul2_rn(A, make_float2(mk.x, mk.y));
    }
    const float4 m = make_float4(A.x, A.y, H.x, H.y);
    if (!CLUSTER) maps.chunk[s & 3][0][lane] = m;
    else
      for (int r = 0; r < cl; ++r) store_cluster_async(&maps.chunk[s & 3][rank][lane], &maps.arrived[s & 3], r, m);
  };
  const auto finish = [&](int s, const float2 (&al)[R], const float2 (&u)[R]) {
    const int j = s * cl + rank, here = min(cl, q.chunks - s * cl);   // chunks of this step
    if (CLUSTER && !mbar_try_wait_cluster(&maps.arrived[s & 3], (s >> 2) & 1) && !lost)
      lost = !wait_longer(&maps.arrived[s & 3], (s >> 2) & 1, a);
    float2 h = x;                                        // the state that enters the block's chunk
    for (int r = 0; r < here; ++r) {
      if (r == rank) h = x;
      x = apply_map(maps.chunk[s & 3][r][lane], x);
    }
    if (j >= q.chunks) return;
    if (a.states && warp == 0) store_io2(a.states + (size_t)(q.chunk0 + j) * a.D + ch, h.x, h.y);
    for (int k = 0; k < warp; ++k) h = apply_map(maps.warp[s & 1][k][lane], h);
    const int n = tokens(s);
    IO* out = static_cast<IO*>(a.out) + (size_t)(q.t0 + j * kChunk + warp * R) * a.D + ch;
    if (n >= R && a.out) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        h = __ffma2_rn(al[i], h, u[i]);
        store_io2(out + (size_t)i * a.D, h.x, h.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          h = __ffma2_rn(al[i], h, u[i]);
          if (a.out) store_io2(out + (size_t)i * a.D, h.x, h.y);
        }
    }
    if (a.hT && n > 0 && j * kChunk + warp * R + n == q.len) store_io2(a.hT + sidx, h.x, h.y);
  };
  // Shared memory: a stage is filled again once every warp has loaded it (the
  // second barrier); maps.warp of step s is written again in step s + 2, after
  // every warp has finished step s (the first barrier of step s + 2); maps.chunk
  // of step s in step s + 4: a block that writes it has finished step s + 2, for
  // which it needed this block's map of that step, which this block hands out
  // after it has finished step s.
  float2 al[2][R], u[2][R];
  const auto step = [&](int s, float2 (&al1)[R], float2 (&u1)[R], const float2 (&al0)[R], const float2 (&u0)[R]) {
    if (s < steps) {
      cp_async_wait<1>();
      __syncthreads();
      load(s, al1, u1);
      __syncthreads();
      fetch(s + 2);
      if (warp == 0) hand_out(s);
    } else if (!CLUSTER) {
      __syncthreads();
    }
    if (s > 0) finish(s - 1, al0, u0);
  };
  for (int s = 0; s <= steps; s += 2) {
    step(s, al[0], u[0], al[1], u[1]);
    if (s < steps) step(s + 1, al[1], u[1], al[0], u[0]);
  }
  if (CLUSTER) end_cluster_walk(lost);
}

// Maps are (A, A', H, H') of a lane's two channels.
struct ScanBwdMaps {
  float4 warp[kScanWarps][32];
  float4 chunk[2][kScanMaxCluster][32];            // by the step's parity, and the rank
  uint64_t arrived[2];                             // the step's maps are here
};

// Backward: one stage of rows in shared memory, filled again once every warp
// has loaded its part and the step's maps are on their way.  (A second stage
// bought nothing: two blocks an SM cover each other's waits, and more reads in
// flight only slow the stores: 165 us against 145 us at 16K x 1 with 16 heads of
// 128.)
template <typename IO, bool CLUSTER>
__global__ void __launch_bounds__(kScanThr, 2) gated_scan_bwd_kernel(const ScanArgs a, int cluster) {
  const int cl = CLUSTER ? cluster : 1;
  constexpr int R = kScanTok, NW = kScanWarps;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  using Stage = ScanStageBwd<IO>;
  Stage& st = *reinterpret_cast<Stage*>(smem_raw);
  __shared__ __align__(128) ScanBwdMaps maps;             // of the gradient's recurrence
  __shared__ float2 wh[kScanWarps][32];                  // H of the warps' maps of the states (A is the same)
  bool lost = false;                                     // a wait of this thread gave up
  const ScanSeq q = scan_seq(a, cl);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rank = CLUSTER ? (int)cluster_rank() : 0;
  const int ch = q.slab * kScanSlab + 2 * lane;
  const size_t sidx = (size_t)q.n * a.D + ch;
  float2 x = make_float2(0.f, 0.f);                      // r that enters the step from the tokens after it
  if (a.dhT) x = load_io2(a.dhT + sidx);
  if (q.len == 0) {
    if (rank == 0 && warp == 0) store_io2(a.dh0 + sidx, x.x, x.y);
    return;
  }
  const int steps = (q.chunks + cl - 1) / cl;
  const auto fetch = [&](int s) {
    const int j = s * cl + rank;
    if (s >= 0 && j < q.chunks) {
      fetch_rows(st.la, a.la, a, q, j);
      fetch_rows(st.w, a.w, a, q, j);
      fetch_rows(st.v, static_cast<const IO*>(a.v), a, q, j);
      fetch_rows(st.dO, static_cast<const IO*>(a.dO), a, q, j);
    }
    cp_async_commit();
  };
  fetch(steps - 1);
  if (CLUSTER) {
    if (threadIdx.x == 0) {
      tc::mbar_init(&maps.arrived[0], 1);
      tc::mbar_init(&maps.arrived[1], 1);
      tc::fence_mbar_init();
    }
    cluster_sync();
  }
  for (int s = steps - 1; s >= 0; --s) {
    const int j = s * cl + rank, here = min(cl, q.chunks - s * cl), k = steps - 1 - s;   // k: steps before this one
    float2 h = make_float2(0.f, 0.f);                    // the state at the chunk's start
    if (j < q.chunks) h = load_io2(a.states + (size_t)(q.chunk0 + j) * a.D + ch);
    cp_async_wait<0>();
    __syncthreads();
    const int n = min(R, min(kChunk, q.len - j * kChunk) - warp * R);
    float2 al[R], w[R], v[R], g[R];
    float2 A = make_float2(1.f, 1.f), H = make_float2(0.f, 0.f), Q = H;
    const auto token = [&](int i) {
      const int r = warp * R + i;
      w[i] = load_io2(&st.w[r][2 * lane]);
      v[i] = load_io2(&st.v[r][2 * lane]);
      g[i] = load_io2(&st.dO[r][2 * lane]);
      al[i] = decay2(load_io2(&st.la[r][2 * lane]));
      A = __fmul2_rn(A, al[i]);
      H = __ffma2_rn(al[i], H, __fmul2_rn(w[i], v[i]));
    };
    if (n >= R) {
#pragma unroll
      for (int i = 0; i < R; ++i) token(i);
#pragma unroll
      for (int i = R - 1; i >= 0; --i) Q = __fmul2_rn(al[i], __fadd2_rn(g[i], Q));
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) token(i);
#pragma unroll
      for (int i = R - 1; i >= 0; --i)
        if (i < n) Q = __fmul2_rn(al[i], __fadd2_rn(g[i], Q));
    }
    maps.warp[warp][lane] = make_float4(A.x, A.y, Q.x, Q.y);
    wh[warp][lane] = H;
    __syncthreads();
    if (CLUSTER && threadIdx.x == 0 && !lost) tc::mbar_arrive_expect_tx(&maps.arrived[k & 1], here * 512u);
    if (warp == 0 && j < q.chunks && !lost) {                     // the chunk's map, to every block of the cluster
      const float4 m0 = maps.warp[NW - 1][lane];
      A = make_float2(m0.x, m0.y);
      Q = make_float2(m0.z, m0.w);
#pragma unroll
      for (int i = NW - 2; i >= 0; --i) {
        const float4 mi = maps.warp[i][lane];
        Q = apply_map(mi, Q);
        A = __fmul2_rn(A, make_float2(mi.x, mi.y));
      }
      const float4 m = make_float4(A.x, A.y, Q.x, Q.y);
      if (!CLUSTER) maps.chunk[k & 1][0][lane] = m;
      else
        for (int r = 0; r < cl; ++r) store_cluster_async(&maps.chunk[k & 1][rank][lane], &maps.arrived[k & 1], r, m);
    }
    // maps.chunk of step k is written again in step k + 2: a block that does so has
    // finished step k + 1, for which it needed this block's map, which this block
    // hands out after it has finished step k.
    if (!CLUSTER) __syncthreads();
    fetch(s - 1);
    if (CLUSTER && !mbar_try_wait_cluster(&maps.arrived[k & 1], (k >> 1) & 1) && !lost)
      lost = !wait_longer(&maps.arrived[k & 1], (k >> 1) & 1, a);
    float2 r2 = x;                                       // r that enters the block's chunk
    for (int r = here - 1; r >= 0; --r) {
      if (r == rank) r2 = x;
      x = apply_map(maps.chunk[k & 1][r][lane], x);
    }
    if (j >= q.chunks) continue;
    for (int i = 0; i < warp; ++i) {
      const float4 mi = maps.warp[i][lane];
      h = __ffma2_rn(make_float2(mi.x, mi.y), h, wh[i][lane]);
    }
    for (int i = NW - 1; i > warp; --i) r2 = apply_map(maps.warp[i][lane], r2);
    float2 p[R];                                         // alpha_t h_{t-1}
    const size_t base = (size_t)(q.t0 + j * kChunk + warp * R) * a.D + ch;
    const auto state = [&](int i) {
      p[i] = __fmul2_rn(al[i], h);
      h = __ffma2_rn(w[i], v[i], p[i]);
    };
    const auto gradient = [&](int i) {
      const size_t at = base + (size_t)i * a.D;
      const float2 gi = __fadd2_rn(g[i], r2), da = __fmul2_rn(p[i], gi), dv = __fmul2_rn(w[i], gi), dw = __fmul2_rn(v[i], gi);
      r2 = __fmul2_rn(al[i], gi);
      store_io2(a.dla + at, da.x, da.y);
      store_io2(a.dv + at, dv.x, dv.y);
      store_io2(a.dw + at, dw.x, dw.y);
    };
    if (n >= R) {
#pragma unroll
      for (int i = 0; i < R; ++i) state(i);
#pragma unroll
      for (int i = R - 1; i >= 0; --i) gradient(i);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) state(i);
#pragma unroll
      for (int i = R - 1; i >= 0; --i)
        if (i < n) gradient(i);
    }
    if (j == 0 && warp == 0) store_io2(a.dh0 + sidx, r2.x, r2.y);
  }
  if (CLUSTER) end_cluster_walk(lost);
}

// One token of n channels (4 per thread), states in place.
constexpr int kStepThr = 128;

template <typename IO>
__global__ void __launch_bounds__(kStepThr)
gated_scan_step_kernel(const void* v, const float* la, const float* w, float* state, void* out, long long n) {
  const long long i = 4 * ((long long)blockIdx.x * kStepThr + threadIdx.x);
  if (i >= n) return;
  float x[4], l[4], g[4], h[4];
  load_vec<4>(static_cast<const IO*>(v) + i, x);
  load_vec<4>(la + i, l);
  load_vec<4>(w + i, g);
  load_vec<4>(state + i, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = fmaf(decay(l[j]), h[j], g[j] * x[j]);
  *reinterpret_cast<float4*>(state + i) = make_float4(h[0], h[1], h[2], h[3]);
  store_io2(static_cast<IO*>(out) + i, h[0], h[1]);
  store_io2(static_cast<IO*>(out) + i + 2, h[2], h[3]);
}

}  // namespace gdn2
