// Test driver for the merge of cut prompt items (pa_prompt_kernel.cuh): its check of the
// entries that say where the partials are, on the host, and the kernel over entries given by
// the test.  Built by tests/test_merge_entries.py.
#include "pa_prompt_kernel.cuh"

using namespace pa;

static PromptParams params(int Hq, int Hkv, int total_q, int grid) {
    PromptParams p{};
    p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
    p.tokens = PT_M / p.G;
    p.total_q = total_q;
    p.grid = grid;
    p.splits = 32;
    return p;
}

extern "C" int merge_parts(int Hq, int Hkv, int total_q, int grid, int i, const int* n, const int* item) {
    return cut_parts(params(Hq, Hkv, total_q, grid), i, make_int4(n[0], n[1], n[2], n[3]),
                     make_int4(item[0], item[1], item[2], item[3]));
}

// f16, head_dim 64; cut holds 1 + grid entries, the partials 2 * grid places.
extern "C" int merge_run(void* out, void* cut, void* part_ml, void* part_acc, int Hq, int Hkv, int total_q, int grid) {
    PromptParams p = params(Hq, Hkv, total_q, grid);
    p.out = out;
    p.cut = static_cast<int4*>(cut);
    p.part_ml = static_cast<float2*>(part_ml);
    p.part_acc = static_cast<float*>(part_acc);
    prompt_merge_kernel<F16T, 64><<<grid * (2 * PT_M / PT_MERGE_ROWS), 32 * PT_MERGE_WARPS>>>(p);
    return static_cast<int>(cudaDeviceSynchronize());
}
