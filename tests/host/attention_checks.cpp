// The C entry points of the attention-side operators against faked launchers:
// sizes at the ends of their ranges, plans that must fit a grid, the propagation
// of HIP errors. Built with the address and undefined-behaviour sanitizers by
// tests/test_attention_host_hardening.py.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include <hip/hip_runtime_api.h>

#include "attn_launch.hpp"
#include "sparse_ffn_attention.h"
#include "status.hpp"

extern hipError_t g_fake_launch_status;
extern int g_fake_launches;
extern sffn::AttnPlan g_fake_plan;

static int g_failed = 0;
static void expect(bool ok, const char* what, int line) {
    if (ok) return;
    std::printf("FAILED line %d: %s (last error: \"%s\")\n", line, what, sffn::last_error);
    ++g_failed;
}
#define EXPECT(cond) expect((cond), #cond, __LINE__)
#define EXPECT_STATUS(call, st) expect((call) == (st), #call " == " #st, __LINE__)

static void* dev(uintptr_t k) { return reinterpret_cast<void*>((uintptr_t)0x10000000u + k * 0x100000u); }

int main() {
    // ---- rotation: sizes whose products pass 31 and 63 bits --------------------
    sffn_rope_config_t r{};
    r.n_q_heads = 32; r.n_k_heads = 8; r.head_dim = 128; r.rot_dim = 128; r.max_pos = INT32_MAX;
    r.dtype = SFFN_BF16; r.layout = SFFN_ROPE_HALF; r.norm = 1; r.eps = 1e-6f;
    const sffn_heads_t q{dev(1), 4096, 128}, wide{dev(2), (int64_t)1 << 42, (int64_t)1 << 42};
    const int32_t* pos = static_cast<int32_t*>(dev(3));
    const float* table = static_cast<float*>(dev(4));
    EXPECT_STATUS(qk_norm_rope(&r, &q, &q, pos, table, nullptr, nullptr, 5, &q, &q, nullptr), SFFN_OK);
    for (int64_t T : {(int64_t)1 << 26, (int64_t)1 << 30, (int64_t)1 << 31, INT64_MAX, INT64_MAX / 40})
        EXPECT_STATUS(qk_norm_rope(&r, &q, &q, pos, table, nullptr, nullptr, T, &q, &q, nullptr), SFFN_ERR_UNSUPPORTED);
    EXPECT_STATUS(qk_norm_rope(&r, &wide, &wide, pos, table, nullptr, nullptr, 1 << 25, &q, &q, nullptr),
                  SFFN_ERR_INVALID_ARG);
    r.n_q_heads = r.n_k_heads = 65536;
    EXPECT_STATUS(qk_norm_rope(&r, &q, &q, pos, table, nullptr, nullptr, 1 << 15, &q, &q, nullptr), SFFN_ERR_UNSUPPORTED);
    r.n_q_heads = 32; r.n_k_heads = 0;
    EXPECT_STATUS(qk_norm_rope(&r, &q, nullptr, pos, table, nullptr, nullptr, 5, &q, nullptr, nullptr), SFFN_OK);
    for (int bad : {INT_MIN, -1, 2, INT_MAX}) {
        sffn_rope_config_t x = r;
        std::memcpy(&x.dtype, &bad, sizeof bad);
        EXPECT_STATUS(qk_norm_rope(&x, &q, nullptr, pos, table, nullptr, nullptr, 5, &q, nullptr, nullptr),
                      SFFN_ERR_INVALID_ARG);
        x = r;
        std::memcpy(&x.layout, &bad, sizeof bad);
        EXPECT_STATUS(qk_norm_rope(&x, &q, nullptr, pos, table, nullptr, nullptr, 5, &q, nullptr, nullptr),
                      SFFN_ERR_INVALID_ARG);
    }
    float* gw = static_cast<float*>(dev(5));
    int before = g_fake_launches;
    EXPECT_STATUS(qk_norm_rope_backward(&r, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0,
                                        nullptr, nullptr, gw, nullptr, nullptr, 0, nullptr), SFFN_OK);
    EXPECT(g_fake_launches == before + 1);          // the zeros of g_q_weight
    EXPECT_STATUS(qk_norm_rope_backward(&r, &q, nullptr, &q, nullptr, pos, table, nullptr, nullptr, 5, &q, nullptr, gw,
                                        nullptr, dev(6), qk_norm_rope_backward_workspace_size(&r, 5), nullptr), SFFN_OK);

    // ---- cache and attention ------------------------------------------------------
    sffn_kv_cache_t c{};
    c.keys = static_cast<int8_t*>(dev(10)); c.values = static_cast<int8_t*>(dev(11));
    c.k_scale = static_cast<float*>(dev(12)); c.v_scale = static_cast<float*>(dev(13));
    c.n_pages = INT32_MAX; c.kv_heads = 8; c.page = 64; c.head_dim = 128;
    sffn_kv_batch_t b{};
    b.block_table = static_cast<int32_t*>(dev(14)); b.kv_lens = static_cast<int32_t*>(dev(15));
    b.cu = static_cast<int32_t*>(dev(16));
    b.n_seqs = 4; b.max_pages = 1000; b.table_stride = 1000; b.max_new = 300; b.max_kv = 60000;
    const sffn_heads_t kv{dev(17), 1024, 128};
    EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, 700, nullptr), SFFN_OK);
    EXPECT_STATUS(kv_cache_read(&c, &b, &kv, &kv, SFFN_F32, 700, nullptr), SFFN_OK);
    // plans over the whole range stay within a grid, and their workspace is what the size says
    for (int heads : {8, 32, 128})
        for (int new_tokens : {0, 1, 2, 5, 17, 300, 1 << 20, INT32_MAX})
            for (int kv_len : {0, 1, 512, 513, 60000, INT32_MAX})
                for (int window : {0, 1, 700, INT32_MAX})
                    for (int64_t T : {(int64_t)1, (int64_t)4, (int64_t)4096, (int64_t)1 << 20}) {
                        sffn_kv_batch_t x = b;
                        x.max_new = new_tokens;
                        x.max_kv = kv_len;
                        const size_t ws = cache_attention_workspace_size(&c, &x, heads, SFFN_BF16, window, T);
                        before = g_fake_launches;
                        const sffn_heads_t h{dev(18), (int64_t)heads * 128, 128};
                        const sffn_status_t st = cache_attention(&c, &x, &h, heads, SFFN_BF16, T, 0.1f, window, &h,
                                                                 nullptr, dev(19), ws, nullptr);
                        EXPECT(st == SFFN_OK || st == SFFN_ERR_UNSUPPORTED);
                        if (g_fake_launches == before) continue;
                        const sffn::AttnPlan& p = g_fake_plan;
                        EXPECT(p.blocks >= 1 && p.blocks < (int64_t)1 << 31 && p.splits >= 1 && p.row_tiles >= 1);
                        EXPECT(p.ws_bytes == ws && (p.splits == 1) == (ws == 0));
                        const int64_t rows = (new_tokens < T ? new_tokens : T) * (heads / 8);
                        EXPECT(p.few == (rows <= 16) && p.row_tiles * p.rows >= rows);
                        EXPECT(p.few || (p.chunk % 64 == 0 && p.chunk >= 64));
                        if (p.splits > 1) {
                            EXPECT_STATUS(cache_attention(&c, &x, &h, heads, SFFN_BF16, T, 0.1f, window, &h, nullptr,
                                                          dev(19), ws - 1, nullptr), SFFN_ERR_WORKSPACE);
                        }
                    }
    const sffn_heads_t h{dev(18), 4096, 128};
    for (int64_t T : {((int64_t)1 << 28) + 1, (int64_t)1 << 40, INT64_MAX}) {
        EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, T, nullptr), SFFN_ERR_UNSUPPORTED);
        EXPECT_STATUS(cache_attention(&c, &b, &h, 32, SFFN_BF16, T, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr),
                      SFFN_ERR_UNSUPPORTED);
        EXPECT(cache_attention_workspace_size(&c, &b, 32, SFFN_BF16, 0, T) == 0);
    }
    sffn_kv_batch_t x = b;
    x.n_seqs = INT32_MAX;
    EXPECT_STATUS(kv_cache_append(&c, &x, &kv, &kv, SFFN_BF16, 700, nullptr), SFFN_ERR_UNSUPPORTED);
    EXPECT_STATUS(cache_attention(&c, &x, &h, 32, SFFN_BF16, 700, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr),
                  SFFN_ERR_UNSUPPORTED);
    x = b;
    x.max_pages = INT32_MAX; x.table_stride = INT32_MAX;
    EXPECT_STATUS(cache_attention(&c, &x, &h, 32, SFFN_BF16, 700, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr),
                  SFFN_ERR_UNSUPPORTED);

    // ---- HIP errors ------------------------------------------------------------------
    g_fake_launch_status = hipErrorLaunchFailure;
    EXPECT_STATUS(qk_norm_rope(&r, &q, nullptr, pos, table, nullptr, nullptr, 5, &q, nullptr, nullptr), SFFN_ERR_HIP);
    EXPECT(std::strstr(sffn::last_error, "qk_norm_rope") != nullptr);
    EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, 700, nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(kv_cache_read(&c, &b, &kv, &kv, SFFN_BF16, 700, nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(cache_attention(&c, &b, &h, 32, SFFN_BF16, 700, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr),
                  SFFN_ERR_HIP);
    EXPECT(std::strstr(sffn::last_error, "cache_attention") != nullptr);

    if (g_failed) {
        std::printf("%d host checks failed\n", g_failed);
        return 1;
    }
    std::printf("host checks passed\n");
    return 0;
}
