/* A C99 caller of every entry point of spec_verify_cache.h, compiled (not
 * run) to check that the header is plain C and complete. */
#include <stddef.h>
#include <stdint.h>

#include "spec_verify_cache.h"

int use_every_cache_entry_point(void *stream)
{
    int32_t *i32 = NULL;
    uint8_t *u8 = NULL;
    const void *cv = NULL;
    void *v = NULL;
    int64_t bytes = 0;
    sv_attention_args a = {0};
    sv_status st = spec_verify_kv_commit_path(cv, v, u8, i32, i32, i32, i32, i32, 56, 256, 8, 1, 2048, 4, 128,
                                              SV_KV_E4M3, stream);
    st = spec_verify_kv_read(v, u8, i32, i32, v, i32, 56, 256, 2048, 2048, 4, 128, stream);
    a.B = 256;
    a.T = 8;
    a.heads_q = 28;
    a.heads_kv = 4;
    a.head_dim = 128;
    a.format = SV_KV_BF16;
    st = spec_verify_attention_workspace(&a, &bytes);
    a.workspace_bytes = bytes;
    st = spec_verify_attention(&a, stream);
    return (int)st + SV_KV_BAD_PATH + SV_KV_NONFINITE + SV_ATTN_BAD_LEN + SV_ATTN_BAD_TREE + SV_ATTN_TIMEOUT;
}
