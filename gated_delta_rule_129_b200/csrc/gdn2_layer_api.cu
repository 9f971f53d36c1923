// gdn2_layer_api.cu -- the C ABI (include/gdn2.h) of what stands around the
// operator in a layer that is trained: 8-bit activation checkpoints, the
// backward passes of the token path, and the gated linear recurrence.
//
// Host side only, as in gdn2_api.cu: argument checks (no CUDA call happens
// before they pass), workspace carving, dispatch.  Nothing here allocates
// device memory or synchronises a stream.
#include "gdn2.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "act_pack.cuh"
#include "api_util.cuh"
#include "common.cuh"
#include "gated_scan.cuh"
#include "plan.cuh"
#include "token_bwd.cuh"

namespace {

using bf16 = __nv_bfloat16;
using gdn2::kChunk;
using namespace gdn2_host;

gdn2_status check_workspace(const gdn2_desc* d, size_t need) {
  if (!d->workspace) return GDN2_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(d->workspace) & (kAlign - 1)) != 0) return GDN2_ERR_ALIGN;
  if (d->workspace_bytes < need) return GDN2_ERR_WORKSPACE;
  return GDN2_OK;
}

bool all_aligned(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned16(p)) return false;
  return true;
}
bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return true;
  return false;
}

// A launch that may begin while the one before it on the stream still runs; it
// waits on the device for that one's end before it reads (after_last_launch).
template <typename... P, typename... A>
gdn2_status launch_after(void (*kern)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  (void)cudaLaunchKernelEx(&c, kern, P(args)...);
  return launch_status();
}

// ------------------------------------------------- activation checkpoints ----
gdn2_status check_pack(long long rows, int cols, gdn2_io_dtype io, const void* x, const void* codes,
                       const void* exps, gdn2::PackArgs* a, int* values, unsigned* grid) {
  if (io != GDN2_IO_F32 && io != GDN2_IO_BF16) return GDN2_ERR_DTYPE;
  if (rows < 0 || cols < 1) return GDN2_ERR_SHAPE;
  if (rows > (1ll << 62) / cols) return GDN2_ERR_SHAPE;
  if (cols % gdn2::kPackCols == 0) {   // whole blocks one after the other
    rows *= cols / gdn2::kPackCols;
    cols = gdn2::kPackCols;
  }
  a->cols = cols;
  a->blocks = cols / gdn2::kPackCols + (cols % gdn2::kPackCols != 0);   // cols may be near 2^31
  if (rows > (1ll << 62) / a->blocks) return GDN2_ERR_SHAPE;
  a->total = rows * a->blocks;
  *values = io == GDN2_IO_BF16 && cols % 8 == 0 ? 8 : 4;   // a lane's
  a->group = 1;
  while (a->group * *values < std::min(cols, gdn2::kPackCols)) a->group *= 2;
  a->step_rows = gdn2::kPackThreads / a->group / a->blocks;
  a->step_blocks = gdn2::kPackThreads / a->group % a->blocks;
  const long long per_cta = gdn2::kPackThreads / a->group * gdn2::kPackPasses;
  const long long ctas = (a->total + per_cta - 1) / per_cta;
  if (ctas > INT32_MAX) return GDN2_ERR_SHAPE;
  if (rows > 0 && any_null({x, codes, exps})) return GDN2_ERR_NULL;
  if (!all_aligned({x, codes, exps})) return GDN2_ERR_ALIGN;
  *grid = (unsigned)ctas;
  return GDN2_OK;
}

// -------------------------------------------------------- token backward ----
// Blocks along the tokens in the prologue's backward pass.  A block's work does
// not depend on how many there are, so the best count fills whole waves of
// blocks: up to four waves, the count that leaves the least of the last wave
// empty, the fewest blocks among equals; and no more than one block for each 64
// tokens begun, so that the W - 1 tokens a warp walks on either side stay few: where
// that limit binds, a warp's run is 9 to 16 tokens (fewer under 65 tokens in all).
constexpr int kProBwdSms = 148;   // B200
constexpr int kProBwdRun = 16;   // tokens of a warp's run at that limit, at most
constexpr int kEpiBwdBlocks = 148 * 4;   // four blocks an SM, each walking rows with a stride

int pro_groups(long long tokens, int rows /* heads times projections of the launch */, int slots) {
  const long long most = std::max<long long>(1, (tokens + gdn2::kBwdWarps * kProBwdRun - 1) / (gdn2::kBwdWarps * kProBwdRun));
  long long best = 1;
  double best_fill = 0;
  for (int waves = 1; waves <= 4; ++waves) {
    const long long g = std::min<long long>(most, std::max<long long>(1, (long long)slots * waves / rows));
    const long long blocks = g * rows, used = (blocks + slots - 1) / slots;
    const double fill = (double)blocks / (double)(used * slots);
    if (fill > best_fill * 1.02) best_fill = fill, best = g;
  }
  return (int)best;
}

struct ProBwdLayout {
  int groups[2];           // of the launch with q and k (and v where dk = dv), of v's own
  size_t off[3], total;
};

// For activations of `bytes` a value (1: 8-bit codes).
gdn2_status pro_bwd_layout(const gdn2_desc* d, bool packed, int W, int bytes, ProBwdLayout* L) {
  gdn2_status st = check_dims(d, packed);
  if (st != GDN2_OK) return st;
  if (W < 1 || W > gdn2::kMaxConvWidth || d->H > 65535) return GDN2_ERR_SHAPE;
  const long long tokens = (long long)d->B * d->T;
  const bool one = d->dk == d->dv;
  const int slots = kProBwdSms * gdn2::pro_bwd_blocks(bytes, W);
  L->groups[0] = pro_groups(tokens, (one ? 3 : 2) * d->H, slots);
  L->groups[1] = one ? L->groups[0] : pro_groups(tokens, d->H, slots);
  size_t off = 0;
  for (int z = 0; z < 3; ++z) {
    L->off[z] = off;
    off = align_up(off + (size_t)L->groups[z == 2] * d->H * (z == 2 ? d->dv : d->dk) * W * sizeof(float));
  }
  L->total = std::max(off, kAlign);
  return GDN2_OK;
}

template <typename XT, typename IO, int D, int W>
gdn2_status launch_pro_bwd_w(const gdn2::TokProBwdArgs& a, dim3 grid, cudaStream_t s) {
  auto kern = gdn2::token_prologue_bwd_kernel<XT, IO, D, W>;
  constexpr int smem = gdn2::pro_bwd_smem<XT>(D, W);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return GDN2_ERR_CUDA;
  kern<<<grid, gdn2::kBwdWarps * 32, smem, s>>>(a);
  return launch_status();
}
template <typename XT, typename IO, int D>
gdn2_status launch_pro_bwd_d(int W, const gdn2::TokProBwdArgs& a, dim3 grid, cudaStream_t s) {
  switch (W) {
    case 1: return launch_pro_bwd_w<XT, IO, D, 1>(a, grid, s);
    case 2: return launch_pro_bwd_w<XT, IO, D, 2>(a, grid, s);
    case 3: return launch_pro_bwd_w<XT, IO, D, 3>(a, grid, s);
    case 4: return launch_pro_bwd_w<XT, IO, D, 4>(a, grid, s);
    case 5: return launch_pro_bwd_w<XT, IO, D, 5>(a, grid, s);
    case 6: return launch_pro_bwd_w<XT, IO, D, 6>(a, grid, s);
    case 7: return launch_pro_bwd_w<XT, IO, D, 7>(a, grid, s);
    case 8: return launch_pro_bwd_w<XT, IO, D, 8>(a, grid, s);
  }
  return GDN2_ERR_SHAPE;
}
template <typename XT, typename IO>
gdn2_status launch_pro_bwd(int d, int W, const gdn2::TokProBwdArgs& a, dim3 grid, cudaStream_t s) {
  return d == 64 ? launch_pro_bwd_d<XT, IO, 64>(W, a, grid, s) : launch_pro_bwd_d<XT, IO, 128>(W, a, grid, s);
}

int epi_bwd_blocks(const gdn2_desc* d) {
  const long long rows = (long long)d->B * d->T * d->H, per = gdn2::kTokThreads * gdn2::kEpiBwdPer / d->dv;
  return (int)std::min<long long>((rows + per - 1) / per, kEpiBwdBlocks);
}

gdn2_status check_epi(const gdn2_desc* d) {
  if (!d) return GDN2_ERR_NULL;
  gdn2_desc e = *d;
  e.num_seqs = 0;   // the epilogue does not look at sequences
  return check_dims(&e, false);
}

template <typename OT, typename GT, typename IO>
void launch_epi_bwd(int dv, const gdn2::TokEpiBwdArgs& a, int blocks, cudaStream_t s) {
  if (dv == 128) gdn2::token_epilogue_bwd_kernel<OT, GT, IO, 128><<<blocks, gdn2::kTokThreads, 0, s>>>(a);
  else gdn2::token_epilogue_bwd_kernel<OT, GT, IO, 64><<<blocks, gdn2::kTokThreads, 0, s>>>(a);
}
template <typename IO>
void dispatch_epi_bwd(int dv, const gdn2::TokEpiBwdArgs& a, int blocks, cudaStream_t s) {
  if (a.o_exps && a.g_exps) launch_epi_bwd<int8_t, int8_t, IO>(dv, a, blocks, s);
  else if (a.o_exps) launch_epi_bwd<int8_t, IO, IO>(dv, a, blocks, s);
  else if (a.g_exps) launch_epi_bwd<IO, int8_t, IO>(dv, a, blocks, s);
  else launch_epi_bwd<IO, IO, IO>(dv, a, blocks, s);
}

// ------------------------------------------------- gated linear recurrence ----
struct ScanLayout {
  int N, max_chunks, D;
  size_t off_status, off_chunk, off_order, total;
};

gdn2_status scan_layout(const gdn2_desc* desc, bool packed, ScanLayout* L) {
  if (!desc) return GDN2_ERR_NULL;
  gdn2_desc d = *desc;
  d.dk = d.dv;   // the recurrence has value channels only
  gdn2_status st = check_dims(&d, packed);
  if (st != GDN2_OK) return st;
  L->N = packed ? d.num_seqs : d.B;
  const long long tokens = (long long)d.B * d.T;
  const long long chunks =
      packed ? tokens / kChunk + L->N : (long long)d.B * ((d.T + kChunk - 1) / kChunk);
  const long long D = (long long)d.H * d.dv;
  // a cluster of blocks per (sequence, slab)
  if (D > INT32_MAX / 2 || L->N * (D / gdn2::kScanSlab) > INT32_MAX / gdn2::kScanMaxCluster) return GDN2_ERR_SHAPE;
  if (chunks > INT32_MAX / 2) return GDN2_ERR_SHAPE;
  L->max_chunks = (int)chunks;
  L->D = (int)D;
  L->off_status = 0;
  L->off_chunk = kAlign;
  L->off_order = align_up(L->off_chunk + (packed ? (size_t)(L->N + 1) * sizeof(int32_t) : 0));
  L->total = align_up(L->off_order + (packed ? (size_t)L->N * sizeof(int32_t) : 0));
  return GDN2_OK;
}

// Blocks per cluster: as many as still let every cluster be resident at once
// at two blocks an SM, and no more than the longest possible sequence has chunks.
int scan_cluster(const gdn2_desc* d, const ScanLayout& L, int most) {
  const long long pairs = (long long)L.N * (L.D / gdn2::kScanSlab), chunks = (d->T + kChunk - 1) / kChunk;
  int cl = 1;
  while (cl < most && pairs * cl * 2 <= 2 * sm_count() && cl < chunks) cl *= 2;
  return cl;
}

// The launch's arguments; calls of many packed sequences check cu_seqlens and
// number the chunks first.
gdn2_status scan_plan(const gdn2_desc* d, const ScanLayout& L, const int32_t* cu, gdn2::ScanArgs* a, cudaStream_t s) {
  a->status = at<int32_t>(d->workspace, L.off_status);
  a->timeout_code = (int)GDN2_ERR_DEVICE_TIMEOUT;
  a->wait_ns = 2000000000ull;
  a->map.cu = cu;
  a->map.N = L.N;
  a->map.T = d->T;
  a->D = L.D;
  a->slabs = L.D / gdn2::kScanSlab;
  a->map.chunk_off = nullptr;
  if (!cu) return GDN2_OK;
  // The longest sequences first, so that none is left for the end when there are
  // more blocks than fit: 32 sequences of 256 to 8192 tokens, 16 heads of 128,
  // 535 -> 447 us forward and 1121 -> 955 us backward.  Not for short sequences
  // (under four chunks on average), which gain nothing.
  const bool sorted = L.N > 1 && d->T / kChunk >= 4 * (long long)L.N;
  if (L.N <= gdn2::kScanLocal) {   // the blocks look at cu_seqlens by themselves
    a->longest_first = sorted;
    a->T_total = d->T;
    a->seqlens_code = (int)GDN2_ERR_SEQLENS;
    return GDN2_OK;
  }
  int32_t* chunk_off = at<int32_t>(d->workspace, L.off_chunk);
  int32_t* order = sorted && L.N <= gdn2::kPlanOrdered ? at<int32_t>(d->workspace, L.off_order) : nullptr;
  gdn2::plan_kernel<<<1, gdn2::kPlanThreads, 0, s>>>(cu, L.N, d->T, d->B * d->T, chunk_off, a->status,
                                                     (int)GDN2_ERR_SEQLENS, nullptr, nullptr, 0, order);
  a->map.chunk_off = chunk_off;
  a->order = order;
  return launch_status();
}

// One of the two forms of a kernel: blocks on their own, or in clusters of cl.
gdn2_status scan_launch(void (*alone)(const gdn2::ScanArgs, int), void (*clustered)(const gdn2::ScanArgs, int),
                        size_t smem, const gdn2::ScanArgs& a, int cl, cudaStream_t s) {
  auto kern = cl == 1 ? alone : clustered;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return GDN2_ERR_CUDA;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(a.map.N * a.slabs * cl));
  c.blockDim = dim3(gdn2::kScanThr);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)cl;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = cl == 1 ? 0 : 1;
  (void)cudaLaunchKernelEx(&c, kern, a, cl);
  return launch_status();
}

}  // namespace

extern "C" {

gdn2_status gdn2_act_pack(const void* x, gdn2_io_dtype io, long long rows, int cols, int8_t* codes, uint8_t* exps,
                          cudaStream_t stream) {
  gdn2::PackArgs a{};
  unsigned grid = 0;
  int values = 0;
  gdn2_status st = check_pack(rows, cols, io, x, codes, exps, &a, &values, &grid);
  if (st != GDN2_OK) return st;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  if (grid == 0) return GDN2_OK;
  a.x = x; a.codes = codes; a.exps = exps;
  const bool vec = a.cols % 4 == 0;
  if (io == GDN2_IO_F32) {
    if (vec) gdn2::act_pack_kernel<float, 4, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else gdn2::act_pack_kernel<float, 4, false><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
  } else {
    if (values == 8) gdn2::act_pack_kernel<bf16, 8, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else if (vec) gdn2::act_pack_kernel<bf16, 4, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else gdn2::act_pack_kernel<bf16, 4, false><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
  }
  return launch_status();
}

gdn2_status gdn2_act_unpack(const int8_t* codes, const uint8_t* exps, long long rows, int cols, gdn2_io_dtype io,
                            void* x, cudaStream_t stream) {
  gdn2::PackArgs a{};
  unsigned grid = 0;
  int values = 0;
  gdn2_status st = check_pack(rows, cols, io, x, codes, exps, &a, &values, &grid);
  if (st != GDN2_OK) return st;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  if (grid == 0) return GDN2_OK;
  a.y = x; a.codes = const_cast<int8_t*>(codes); a.exps = const_cast<uint8_t*>(exps);
  const bool vec = a.cols % 4 == 0;
  if (io == GDN2_IO_F32) {
    if (vec) gdn2::act_unpack_kernel<float, 4, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else gdn2::act_unpack_kernel<float, 4, false><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
  } else {
    if (values == 8) gdn2::act_unpack_kernel<bf16, 8, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else if (vec) gdn2::act_unpack_kernel<bf16, 4, true><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
    else gdn2::act_unpack_kernel<bf16, 4, false><<<grid, gdn2::kPackThreads, 0, stream>>>(a);
  }
  return launch_status();
}

size_t gdn2_token_prologue_bwd_workspace_size(const gdn2_desc* desc, int conv_width) {
  if (!desc) return 0;
  ProBwdLayout L, L8;   // enough for either form of the activations
  const int bytes = desc->io == GDN2_IO_F32 ? 4 : 2;
  if (pro_bwd_layout(desc, desc->num_seqs > 0, conv_width, bytes, &L) != GDN2_OK) return 0;
  if (pro_bwd_layout(desc, desc->num_seqs > 0, conv_width, 1, &L8) != GDN2_OK) return 0;
  return std::max(L.total, L8.total);
}

gdn2_status gdn2_token_prologue_bwd(const gdn2_desc* desc, const void* q_raw, const void* k_raw, const void* v_raw,
                                    const uint8_t* q_exps, const uint8_t* k_exps, const uint8_t* v_exps,
                                    const float* conv_q, const float* conv_k, const float* conv_v, int conv_width,
                                    const int32_t* cu_seqlens, const float* dq, const float* dk, const float* dv,
                                    void* dq_raw, void* dk_raw, void* dv_raw, float* dconv_q, float* dconv_k,
                                    float* dconv_v, cudaStream_t stream) {
  if (!desc) return GDN2_ERR_NULL;
  ProBwdLayout L;
  const bool x8 = q_exps != nullptr;
  gdn2_status st = pro_bwd_layout(desc, cu_seqlens != nullptr, conv_width, x8 ? 1 : desc->io == GDN2_IO_F32 ? 4 : 2, &L);
  if (st != GDN2_OK) return st;
  if ((st = check_workspace(desc, gdn2_token_prologue_bwd_workspace_size(desc, conv_width))) != GDN2_OK) return st;
  const long long tokens = (long long)desc->B * desc->T;
  if (any_null({conv_q, conv_k, conv_v, dconv_q, dconv_k, dconv_v})) return GDN2_ERR_NULL;
  if (tokens > 0 && any_null({q_raw, k_raw, v_raw, dq, dk, dv, dq_raw, dk_raw, dv_raw})) return GDN2_ERR_NULL;
  if ((k_exps != nullptr) != x8 || (v_exps != nullptr) != x8) return GDN2_ERR_NULL;
  if (!all_aligned({q_raw, k_raw, v_raw, q_exps, k_exps, v_exps, conv_q, conv_k, conv_v, dq, dk, dv, dq_raw, dk_raw,
                    dv_raw, dconv_q, dconv_k, dconv_v}))
    return GDN2_ERR_ALIGN;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  const size_t tk = (size_t)desc->H * desc->dk * conv_width, tv = (size_t)desc->H * desc->dv * conv_width;
  if (tokens == 0) {
    if (cudaMemsetAsync(dconv_q, 0, tk * sizeof(float), stream) != cudaSuccess ||
        cudaMemsetAsync(dconv_k, 0, tk * sizeof(float), stream) != cudaSuccess ||
        cudaMemsetAsync(dconv_v, 0, tv * sizeof(float), stream) != cudaSuccess)
      return GDN2_ERR_CUDA;
    return GDN2_OK;
  }
  const bool f32 = desc->io == GDN2_IO_F32;
  gdn2::TokProBwdArgs a{};
  a.cu = cu_seqlens;
  a.N = cu_seqlens ? desc->num_seqs : desc->B;
  a.T = desc->T;
  a.T_total = (int)tokens;
  a.H = desc->H;
  const auto set = [&](gdn2::TokProBwdArgs& b, int z, const void* x, const uint8_t* ex, const float* wt,
                       const float* dy, void* dx, size_t off, int l2) {
    b.x[z] = x; b.exps[z] = ex; b.wt[z] = wt; b.dy[z] = dy; b.dx[z] = dx;
    b.part[z] = at<float>(desc->workspace, off);
    b.l2[z] = l2;
  };
  set(a, 0, q_raw, q_exps, conv_q, dq, dq_raw, L.off[0], 1);
  set(a, 1, k_raw, k_exps, conv_k, dk, dk_raw, L.off[1], 1);
  gdn2::TokProBwdArgs av = a;
  const bool one = desc->dk == desc->dv;
  set(one ? a : av, one ? 2 : 0, v_raw, v_exps, conv_v, dv, dv_raw, L.off[2], 0);
  const auto launch = [&](int d, gdn2::TokProBwdArgs& b, int groups, int z) {
    const dim3 g((unsigned)groups, (unsigned)desc->H, (unsigned)z);
    b.run = (int)((tokens + (long long)groups * gdn2::kBwdWarps - 1) / ((long long)groups * gdn2::kBwdWarps));
    if (x8 && f32) return launch_pro_bwd<int8_t, float>(d, conv_width, b, g, stream);
    if (x8) return launch_pro_bwd<int8_t, bf16>(d, conv_width, b, g, stream);
    if (f32) return launch_pro_bwd<float, float>(d, conv_width, b, g, stream);
    return launch_pro_bwd<bf16, bf16>(d, conv_width, b, g, stream);
  };
  if ((st = launch(desc->dk, a, L.groups[0], one ? 3 : 2)) != GDN2_OK) return st;
  if (!one && (st = launch(desc->dv, av, L.groups[1], 1)) != GDN2_OK) return st;
  gdn2::SumPartsArgs s{};
  const size_t n[3] = {tk, tk, tv};
  float* y[3] = {dconv_q, dconv_k, dconv_v};
  for (int z = 0; z < 3; ++z) {
    s.part[z] = at<float>(desc->workspace, L.off[z]);
    s.y[z] = y[z];
    s.n[z] = (int)n[z];
    s.groups[z] = L.groups[z == 2];
  }
  const unsigned bx = (unsigned)((std::max(tk, tv) + gdn2::kTokThreads - 1) / gdn2::kTokThreads);
  return launch_after(gdn2::sum_parts_kernel, dim3(bx, 3), gdn2::kTokThreads, stream, s);
}

size_t gdn2_token_epilogue_bwd_workspace_size(const gdn2_desc* desc) {
  if (check_epi(desc) != GDN2_OK) return 0;
  return std::max(kAlign, align_up((size_t)epi_bwd_blocks(desc) * desc->dv * sizeof(float)));
}

gdn2_status gdn2_token_epilogue_bwd(const gdn2_desc* desc, const void* o, const uint8_t* o_exps, const void* gate,
                                    const uint8_t* gate_exps, const float* norm_weight, const void* dout, void* d_o,
                                    void* d_gate, float* d_norm_weight, cudaStream_t stream) {
  gdn2_status st = check_epi(desc);
  if (st != GDN2_OK) return st;
  if ((st = check_workspace(desc, gdn2_token_epilogue_bwd_workspace_size(desc))) != GDN2_OK) return st;
  const long long tokens = (long long)desc->B * desc->T;
  if (any_null({norm_weight, d_norm_weight})) return GDN2_ERR_NULL;
  if (tokens > 0 && any_null({o, gate, dout, d_o, d_gate})) return GDN2_ERR_NULL;
  if (!all_aligned({o, o_exps, gate, gate_exps, norm_weight, dout, d_o, d_gate, d_norm_weight})) return GDN2_ERR_ALIGN;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  if (tokens == 0)
    return cudaMemsetAsync(d_norm_weight, 0, desc->dv * sizeof(float), stream) == cudaSuccess ? GDN2_OK : GDN2_ERR_CUDA;
  gdn2::TokEpiBwdArgs a{};
  a.o = o; a.g = gate; a.o_exps = o_exps; a.g_exps = gate_exps;
  a.weight = norm_weight; a.dout = dout; a.d_o = d_o; a.d_g = d_gate;
  a.part = at<float>(desc->workspace, 0);
  a.rows = tokens * desc->H;
  const int blocks = epi_bwd_blocks(desc);
  if (desc->io == GDN2_IO_F32) dispatch_epi_bwd<float>(desc->dv, a, blocks, stream);
  else dispatch_epi_bwd<bf16>(desc->dv, a, blocks, stream);
  if ((st = launch_status()) != GDN2_OK) return st;
  return launch_after(gdn2::sum_weight_kernel, dim3(desc->dv / gdn2::kSumCols), 256, stream,
                      (const float*)a.part, blocks, desc->dv, d_norm_weight);
}

size_t gdn2_gated_scan_workspace_size(const gdn2_desc* desc) {
  ScanLayout L;
  if (!desc || scan_layout(desc, desc->num_seqs > 0, &L) != GDN2_OK) return 0;
  return L.total;
}

gdn2_status gdn2_gated_scan_fwd(const gdn2_desc* desc, const void* v, const float* log_alpha, const float* w,
                                const float* h0, const int32_t* cu_seqlens, void* out, float* hT,
                                float* chunk_states, cudaStream_t stream) {
  ScanLayout L;
  gdn2_status st = scan_layout(desc, cu_seqlens != nullptr, &L);
  if (st != GDN2_OK) return st;
  if ((st = check_workspace(desc, L.total)) != GDN2_OK) return st;
  const long long tokens = (long long)desc->B * desc->T;
  if (tokens > 0 && any_null({v, log_alpha, w})) return GDN2_ERR_NULL;
  if (!all_aligned({v, log_alpha, w, h0, out, hT, chunk_states})) return GDN2_ERR_ALIGN;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  gdn2::ScanArgs a{};
  if ((st = scan_plan(desc, L, cu_seqlens, &a, stream)) != GDN2_OK) return st;
  a.v = v; a.la = log_alpha; a.w = w; a.h0 = h0;
  a.out = out; a.hT = hT; a.states = chunk_states;
  if (desc->io == GDN2_IO_F32)
    return scan_launch(gdn2::gated_scan_fwd_kernel<float, false>, gdn2::gated_scan_fwd_kernel<float, true>, 2 * sizeof(gdn2::ScanStageFwd<float>), a,
                       scan_cluster(desc, L, gdn2::scan_max_cluster<float>()), stream);
  return scan_launch(gdn2::gated_scan_fwd_kernel<bf16, false>, gdn2::gated_scan_fwd_kernel<bf16, true>, 2 * sizeof(gdn2::ScanStageFwd<bf16>), a,
                     scan_cluster(desc, L, gdn2::scan_max_cluster<bf16>()), stream);
}

gdn2_status gdn2_gated_scan_bwd(const gdn2_desc* desc, const void* v, const float* log_alpha, const float* w,
                                const float* chunk_states, const int32_t* cu_seqlens, const void* dO,
                                const float* dhT, float* dv, float* dlog_alpha, float* dw, float* dh0,
                                cudaStream_t stream) {
  ScanLayout L;
  gdn2_status st = scan_layout(desc, cu_seqlens != nullptr, &L);
  if (st != GDN2_OK) return st;
  if ((st = check_workspace(desc, L.total)) != GDN2_OK) return st;
  const long long tokens = (long long)desc->B * desc->T;
  if (tokens > 0 && any_null({v, log_alpha, w, chunk_states, dO, dv, dlog_alpha, dw})) return GDN2_ERR_NULL;
  if (!dh0) return GDN2_ERR_NULL;
  if (!all_aligned({v, log_alpha, w, chunk_states, dO, dhT, dv, dlog_alpha, dw, dh0})) return GDN2_ERR_ALIGN;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  gdn2::ScanArgs a{};
  if ((st = scan_plan(desc, L, cu_seqlens, &a, stream)) != GDN2_OK) return st;
  a.v = v; a.la = log_alpha; a.w = w; a.states = const_cast<float*>(chunk_states);
  a.dO = dO; a.dhT = dhT;
  a.dv = dv; a.dla = dlog_alpha; a.dw = dw; a.dh0 = dh0;
  const int cl = scan_cluster(desc, L, gdn2::kScanMaxCluster);
  if (desc->io == GDN2_IO_F32)
    return scan_launch(gdn2::gated_scan_bwd_kernel<float, false>, gdn2::gated_scan_bwd_kernel<float, true>, sizeof(gdn2::ScanStageBwd<float>), a, cl, stream);
  return scan_launch(gdn2::gated_scan_bwd_kernel<bf16, false>, gdn2::gated_scan_bwd_kernel<bf16, true>, sizeof(gdn2::ScanStageBwd<bf16>), a, cl, stream);
}

gdn2_status gdn2_gated_scan_step(const gdn2_desc* desc, const void* v, const float* log_alpha, const float* w,
                                 float* state, void* out, cudaStream_t stream) {
  if (!desc) return GDN2_ERR_NULL;
  if (desc->io != GDN2_IO_F32 && desc->io != GDN2_IO_BF16) return GDN2_ERR_DTYPE;
  if ((desc->dv != 64 && desc->dv != 128) || desc->B < 0 || desc->H < 1) return GDN2_ERR_SHAPE;
  const long long n = (long long)desc->B * desc->H * desc->dv;
  const long long blocks = (n / 4 + gdn2::kStepThr - 1) / gdn2::kStepThr;
  if ((long long)desc->B * desc->H > INT32_MAX) return GDN2_ERR_SHAPE;
  if (n > 0 && any_null({v, log_alpha, w, state, out})) return GDN2_ERR_NULL;
  if (!all_aligned({v, log_alpha, w, state, out})) return GDN2_ERR_ALIGN;
  if (!device_ok()) return GDN2_ERR_UNSUPPORTED;
  if (n == 0) return GDN2_OK;
  if (desc->io == GDN2_IO_F32)
    gdn2::gated_scan_step_kernel<float><<<(unsigned)blocks, gdn2::kStepThr, 0, stream>>>(v, log_alpha, w, state, out, n);
  else
    gdn2::gated_scan_step_kernel<bf16><<<(unsigned)blocks, gdn2::kStepThr, 0, stream>>>(v, log_alpha, w, state, out, n);
  return launch_status();
}

}  // extern "C"
