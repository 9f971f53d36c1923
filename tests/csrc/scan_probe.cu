// scan_probe.cu -- test-only launches of the gated scan's cluster kernels with a
// limit of one's own for their waits, and with blocks whose maps never come.
//
// LONE: the hardware cluster has twice the blocks that the walk counts on, so its
// upper half is the walk of a second slab whose maps all go to the lower half's
// blocks (ranks below `cl`): no block of the upper half ever receives one, and its
// waits can only run out.  Every address stays in bounds: an upper rank indexes the
// maps' places below the largest cluster, its chunks are those of its own slab with
// j < chunks, and no block stores to a rank that is not there.  The lower blocks'
// barriers count the bytes of at most two steps too many, so that their maps mean
// nothing, but each of their phases is still armed once and by a thread that saw
// the one before complete.  Every wait ends by its limit, and every block reaches
// the cluster's last barrier, long after the last store to it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gated_scan.cuh"

using namespace gdn2;

namespace {

template <typename Stage>
int launch(void (*kern)(const ScanArgs, int), int stages, const ScanArgs& a, int cl, int hw, cudaStream_t s) {
  const int smem = stages * (int)sizeof(Stage);
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(a.map.N * a.slabs * cl));
  c.blockDim = dim3(kScanThr);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)hw;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  c.attrs = &attr;
  c.numAttrs = 1;
  (void)cudaLaunchKernelEx(&c, kern, a, cl);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}

}  // namespace

// One sequence of T tokens, D channels; f32: the type of v, dO and out.
extern "C" int scan_probe(int backward, int f32, int lone, int cl, unsigned long long wait_ns, int T, int D, const void* v,
                          const float* la, const float* w, const void* dO, void* out, float* hT, float* states, float* dv,
                          float* dla, float* dw, float* dh0, int* status, void* stream) {
  const int most = backward ? kScanMaxCluster : f32 ? scan_max_cluster<float>() : scan_max_cluster<__nv_bfloat16>();
  const int hw = lone ? 2 * cl : cl;
  if (cl < 2 || hw > most || D % kScanSlab != 0 || (D / kScanSlab * cl) % hw != 0) return 2;
  ScanArgs a{};
  a.v = v; a.la = la; a.w = w; a.dO = dO;
  a.out = out; a.hT = hT; a.states = states;
  a.dv = dv; a.dla = dla; a.dw = dw; a.dh0 = dh0;
  a.map.N = 1;
  a.map.T = T;
  a.D = D;
  a.slabs = D / kScanSlab;
  a.status = status;
  a.timeout_code = 8;
  a.wait_ns = wait_ns;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (backward)
    return f32 ? launch<ScanStageBwd<float>>(gated_scan_bwd_kernel<float, true>, 1, a, cl, hw, s)
               : launch<ScanStageBwd<__nv_bfloat16>>(gated_scan_bwd_kernel<__nv_bfloat16, true>, 1, a, cl, hw, s);
  return f32 ? launch<ScanStageFwd<float>>(gated_scan_fwd_kernel<float, true>, 2, a, cl, hw, s)
             : launch<ScanStageFwd<__nv_bfloat16>>(gated_scan_fwd_kernel<__nv_bfloat16, true>, 2, a, cl, hw, s);
}
