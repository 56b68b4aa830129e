// Stands in for the kernels behind ac_layer.cu (cudart_stub.c for the CUDA
// runtime), so that its argument checks run on a machine without a GPU.  Each
// launcher only counts and keeps what it was given.
#include "ac_layer.cuh"

static int g_launches;
static ac::RowArgs g_rows;
static ac::BackArgs g_back;
static ac::CacheAttnArgs g_attn;
static ac::FreqArgs g_freq;

extern "C" {
__attribute__((visibility("default"))) int stub_launches() { return g_launches; }
__attribute__((visibility("default"))) double stub_freq(int i) { return i < 0 ? g_freq.mag : g_freq.f[i]; }
// q rows of the last ac_qk_norm_rope / ac_cache_append, its paging and its tensors
__attribute__((visibility("default"))) int stub_rows(int what) {
    const int v[] = {g_rows.nt,          g_rows.batch,         g_rows.n,           g_rows.page.seqs,
                     g_rows.page.page_log2, g_rows.rope.pairs, g_rows.rope.cells, (int)g_rows.rope.off[1],
                     (int)g_rows.rope.off[2]};
    return v[what];
}
__attribute__((visibility("default"))) int stub_attn(int what) {
    const int v[] = {g_attn.max_q, g_attn.max_kv, g_attn.group, g_attn.page_log2, g_attn.causal_block, g_attn.window};
    return v[what];
}
}

namespace ac {
void note_launch() {}
int rope_setup(int, int, int, int) { return 0; }
int cache_attn_setup(int) { return 0; }
size_t cache_attn_ws(int, int) { return 4096; }
int back_ctas(int) { return 8; }
void k_rope_table(const RopeArgs &, const FreqArgs &f, float2 *, cudaStream_t) { g_freq = f, g_launches++; }
int k_norm_rope(const RowArgs &a, int, int, int, cudaStream_t) { return g_rows = a, g_launches++, 0; }
int k_norm_rope_back(BackArgs &a, int, int, int, cudaStream_t) { return g_back = a, g_launches++, 0; }
int k_cache_attn(const CacheAttnArgs &a, int, void *, cudaStream_t) { return g_attn = a, g_launches++, 0; }
}  // namespace ac
