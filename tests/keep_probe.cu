// Keeping a long sequence's tokens where the first segments' steps never come: the step
// that waits for them runs out of time, is recorded and leaves its tokens where they are;
// the ones behind it go on.  One CTA: of several, those that wait for what another has
// behind its late step may run out of time as well.
#include "../bit_quantized_kv_02_gb300/csrc/kvq_pages_branch.cu"

using namespace kvq;

// One sequence over fp16 pages of 16 tokens, one head of 64: `pool` [pages][4096 bytes].
// `skip`: segments whose steps are not drawn by anyone (each is one step here).  Device
// pointers; work: pages_keep_bytes(), which keep_probe_bytes gives.
extern "C" size_t keep_probe_bytes() { return pages_keep_bytes(); }
extern "C" int keep_probe(void* pool, int pages, const int* q_start, const int* lens, const int* table, int rows,
                          const uint8_t* keep, int skip, unsigned long long limit, int* lens_out, void* work, int* err) {
  PagesView pv = {};
  pv.base = static_cast<char*>(pool);
  pv.L.k_bits = pv.L.v_bits = 16;
  pv.L.km_off = pv.L.v_off = 2048;
  pv.L.vm_off = pv.L.tile_bytes = 4096;
  pv.pages = pages, pv.heads = 1, pv.head_dim = 64, pv.lg_pt = 4;
  pv.err = err;
  BatchView bv = {1, rows, q_start, lens, table, pages};
  long layer_bytes = 4096L * pages, units = columns(pv);
  KeepPlan* plan = static_cast<KeepPlan*>(work);
  KeepSeg* seg = reinterpret_cast<KeepSeg*>(static_cast<char*>(work) + 256);
  if (units > 32 || (rows + kSegRows - 1) / kSegRows > kKeepSegs) return -1;
  void* args1[] = {&pv, &bv, &keep, &lens_out, &plan, &seg};
  cudaError_t e = launch_pdl((const void*)pages_keep_plan_kernel, dim3(1), dim3(kPlanThreads), 0, nullptr, args1);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  const unsigned long long ticket = skip;
  if (e == cudaSuccess) e = cudaMemcpy(&plan->ticket, &ticket, sizeof(ticket), cudaMemcpyHostToDevice);
  void* args2[] = {&pv, &layer_bytes, &units, &bv, &keep, &plan, &seg, &limit};
  if (e == cudaSuccess) e = launch_pdl((const void*)pages_keep_move_kernel, dim3(1), dim3(kKeepThreads), 0, nullptr, args2);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  return (int)e;
}
