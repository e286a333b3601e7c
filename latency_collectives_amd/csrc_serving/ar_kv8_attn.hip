// Host side of the 8-bit paged cache: the handle and the attention's launch, both as for the 4-bit one.

#include "ar_kv8.h"

namespace ard {

AttnKernel select_attn8_bf16(int head_dim, int columns);
AttnKernel select_attn8_f32(int head_dim, int columns);
AttnKernel select_attn8_rows(int head_dim, bool brief);

static const AttnFormat kFormat8 = {select_attn8_bf16, select_attn8_f32, select_attn8_rows, true,
                                    [](const ar_kv4* h) { return int64_t(2) * h->heads * h->page_size * h->head_dim; },
                                    [](const ar_kv4* h) { return int64_t(2) * h->heads * (h->page_size / kBlock); }};

}  // namespace ard

extern "C" {

ar_kv8* ar_kv8_create(int kv_heads, int head_dim, int page_size) {
  return static_cast<ar_kv8*>(ard::create_handle(ard::kFormat8, kv_heads, head_dim, page_size, "ar_kv8_create"));
}

void ar_kv8_destroy(ar_kv8* h) { ar_kv4_destroy(h); }

int ar_kv8_attention(ar_kv8* h, const ar_kv8_attention_args* a, void* stream) {
  return ard::launch_attention(ard::kFormat8, h, a, stream);
}

}  // extern "C"
