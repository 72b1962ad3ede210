// Further tests on a host without a GPU, of the calls around the paged cache
// in a decoding step: hip_stub.cpp's HIP with a program of its own.
//
// usage: step_stub <test>; prints what the test looks at.
#define main stub_main
#include "hip_stub.cpp"
#undef main

static int sample(int64_t rows, int64_t cols, float top_p,
                  libtopk_stream_t s) {
  libtopk_sampling_t how = {};
  how.temperature_all = 1.0f;
  how.top_p_all = top_p;
  // (so many logits span more than the fake addresses are apart)
  return sample_logits((void*)((uintptr_t)1 << 50), LIBTOPK_F32, rows, cols,
                       cols, &how, fake<float>(0), fake<int64_t>(1),
                       fake<float>(2), s);
}

// Sampling of two sizes and attention share a stream's workspace.
static int step_threads_test() {
  const libtopk_cache_t c = cache_of(2, 4, 256, 64);
  const libtopk_ledger_t l = ledger_of(160, 4, 4096);
  return threads_test(3, [&](int i) {
    return i == 0   ? sample(3, 5000, 0.9f, nullptr)
           : i == 1 ? sample(40, 131072 * (this_call % 2 + 1), 0.9f, nullptr)
                    : attend(c, 16, &l, nullptr);
  });
}

// Launches of one call, the most workgroups and the most threads of one.
static int sample_test(int64_t rows, int64_t cols, float top_p) {
  // (the first call clears a workspace, too)
  if (sample(rows, cols, top_p, nullptr) != LIBTOPK_OK) return 1;
  launches.clear();
  const int rc = sample(rows, cols, top_p, nullptr);
  uint64_t groups = 0, threads = 0;
  for (const Launch& x : launches) {
    const uint64_t t = (uint64_t)x.grid.x * x.block.x;
    groups = x.grid.x > groups ? x.grid.x : groups;
    threads = t > threads ? t : threads;
  }
  // (workspaces are handed out one after the other)
  printf("rc %d launches %zu groups %llu wide %d bytes %llu\n", rc,
         launches.size(), (unsigned long long)groups, threads >> 32 != 0,
         (unsigned long long)(next_address - ((uintptr_t)1 << 40)));
  return 0;
}

// An extension of a 4-bit cache by `tokens` tokens of `batch` sequences.
static int extend_test(int batch, int tokens, int q_heads, int heads) {
  libtopk_cache_t c = cache_of(batch, heads, 4, 64);
  c.dtype = LIBTOPK_E2M1;
  c.k_slot_stride = c.v_slot_stride = 32;
  c.k_head_stride = c.v_head_stride = 16 * 32;
  c.k_page_stride = c.v_page_stride = (int64_t)heads * 16 * 32;
  c.k_block_slot_stride = c.v_block_slot_stride = 2;
  c.k_block_head_stride = c.v_block_head_stride = 16 * 2;
  c.k_block_page_stride = c.v_block_page_stride = heads * 16 * 2;
  c.pages = 64;
  c.k_blocks = fake<char>(100);
  c.v_blocks = fake<char>(101);
  libtopk_tokens_t t = {};
  t.k = (void*)((uintptr_t)1 << 50);
  t.v = (void*)((uintptr_t)1 << 51);
  t.q = (void*)((uintptr_t)1 << 52);
  t.q_out = (void*)((uintptr_t)1 << 53);
  t.k_head_stride = t.v_head_stride = t.q_head_stride = t.q_out_head_stride =
      64;
  t.k_token_stride = t.v_token_stride = (int64_t)heads * 64;
  t.q_token_stride = t.q_out_token_stride = (int64_t)q_heads * 64;
  t.starts = (int32_t*)((uintptr_t)1 << 54);
  t.tokens = tokens;
  t.q_heads = q_heads;
  t.dtype = LIBTOPK_BF16;
  c.table = (int32_t*)((uintptr_t)1 << 55);
  c.lens = (int32_t*)((uintptr_t)1 << 56);
  const int rc = cache_extend(&c, &t, nullptr, (int32_t*)((uintptr_t)1 << 57),
                              nullptr);
  printf("rc %d launches %zu groups %u\n", rc, launches.size(),
         launches.empty() ? 0 : launches[0].grid.x);
  return 0;
}

int main(int n, char** a) {
  const std::string what = n > 1 ? a[1] : "";
  if (what == "threads") return step_threads_test();
  if (what == "sample" && n > 4)
    return sample_test(atoll(a[2]), atoll(a[3]), (float)atof(a[4]));
  if (what == "extend" && n > 5)
    return extend_test(atoi(a[2]), atoi(a[3]), atoi(a[4]), atoi(a[5]));
  return 2;
}
