// The launchers of the attention-side operators against a faked HIP runtime that
// records every launch: whatever size the entry points accept, each launch keeps to
// HIP's limit (fewer than 2^32 threads in a grid) and all of them together cover the
// work; a batch with one long prompt is not launched for prompts of all its
// sequences. Built and run by tests/test_attention_launch_limits.py.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include <hip/hip_runtime.h>

#include "attn_launch.hpp"
#include "sparse_ffn_attention.h"
#include "status.hpp"

alignas(256) unsigned char fake_fatbin[64];

struct Launch {
    uint64_t blocks, threads;
};
static std::vector<Launch> g_launches;
static dim3 g_grid, g_block;

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* h = nullptr; return &h; }
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t, hipStream_t) {
    g_grid = grid;
    g_block = block;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3* grid, dim3* block, size_t* shmem, hipStream_t* s) {
    *grid = g_grid;
    *block = g_block;
    *shmem = 0;
    *s = nullptr;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void*, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    g_launches.push_back({(uint64_t)grid.x * grid.y * grid.z, (uint64_t)block.x * block.y * block.z});
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "HIP error"; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
}
namespace sffn {
hipError_t launch_zero_f32(float*, int64_t, hipStream_t) { return hipSuccess; }
}

static int g_failed = 0;
static void expect(bool ok, const char* what, int line) {
    if (ok) return;
    std::printf("FAILED line %d: %s (last error: \"%s\")\n", line, what, sffn::last_error);
    ++g_failed;
}
#define EXPECT(cond) expect((cond), #cond, __LINE__)
#define EXPECT_STATUS(call, st) expect((call) == (st), #call " == " #st, __LINE__)

static void* dev(uintptr_t k) { return reinterpret_cast<void*>((uintptr_t)0x10000000u + k * 0x100000u); }

// Launches since the last call: all within the limit; workgroups in all.
static uint64_t launched(int line) {
    uint64_t sum = 0;
    for (const Launch& l : g_launches) {
        expect(l.blocks >= 1 && l.blocks * l.threads < (uint64_t)1 << 32, "a grid of fewer than 2^32 threads", line);
        sum += l.blocks;
    }
    g_launches.clear();
    return sum;
}
#define LAUNCHED() launched(__LINE__)

int main() {
    // ---- rotation: wide rows, and heads that go element by element -----------------
    sffn_rope_config_t r{};
    r.n_q_heads = 32; r.n_k_heads = 8; r.rot_dim = 8; r.max_pos = 1000;
    r.dtype = SFFN_BF16; r.layout = SFFN_ROPE_INTERLEAVED; r.norm = 0; r.eps = 1e-6f;
    const int32_t* pos = static_cast<int32_t*>(dev(3));
    const float* table = static_cast<float*>(dev(4));
    for (int dim : {8, 64, 65, 80, 128, 256, 512})
        for (int64_t T : {(int64_t)1, (int64_t)1 << 15, (int64_t)1 << 21, (int64_t)50000000})
            for (int norm : {0, 1}) {
                r.head_dim = dim;
                r.norm = norm;
                const sffn_heads_t q{dev(1), 40 * dim, dim};
                EXPECT_STATUS(qk_norm_rope(&r, &q, &q, pos, table, nullptr, nullptr, T, &q, &q, nullptr), SFFN_OK);
                EXPECT(LAUNCHED() >= 1);
                EXPECT_STATUS(qk_norm_rope_backward(&r, &q, &q, &q, &q, pos, table, nullptr, nullptr, T, &q, &q,
                                                    nullptr, nullptr, nullptr, 0, nullptr), SFFN_OK);
                EXPECT(LAUNCHED() >= 1);
            }

    // ---- append and read ------------------------------------------------------------
    sffn_kv_cache_t c{};
    c.keys = static_cast<int8_t*>(dev(10)); c.values = static_cast<int8_t*>(dev(11));
    c.k_scale = static_cast<float*>(dev(12)); c.v_scale = static_cast<float*>(dev(13));
    c.n_pages = INT32_MAX; c.kv_heads = 8; c.page = 16; c.head_dim = 128;
    sffn_kv_batch_t b{};
    b.block_table = static_cast<int32_t*>(dev(14)); b.kv_lens = static_cast<int32_t*>(dev(15));
    b.cu = static_cast<int32_t*>(dev(16));
    b.n_seqs = 256; b.max_pages = 8192; b.table_stride = 8192; b.max_new = 131072; b.max_kv = 131072;
    const sffn_heads_t kv{dev(17), 1024, 128};
    // 255 single tokens beside a prompt of 131072: of 33.6 million (sequence, page, head)
    // places of keys and values 135 thousand have tokens
    const int64_t T = 131072 + 255;
    EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, T, nullptr), SFFN_OK);
    uint64_t n = LAUNCHED();
    EXPECT(n >= 131072 / 16 * 16 && n < 200000);
    EXPECT_STATUS(kv_cache_read(&c, &b, &kv, &kv, SFFN_BF16, T, nullptr), SFFN_OK);
    n = LAUNCHED();
    EXPECT(n >= 131072 / 16 * 16 && n < 200000);
    // a decode step and a chunk alone: a workgroup for each page that can hold a token
    b.max_new = 1;
    EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, 256, nullptr), SFFN_OK);
    EXPECT(LAUNCHED() == 256 * 8 * 2);
    b.n_seqs = 1; b.max_new = 4095;
    EXPECT_STATUS(kv_cache_append(&c, &b, &kv, &kv, SFFN_BF16, 4095, nullptr), SFFN_OK);
    EXPECT(LAUNCHED() == 257 * 8 * 2);
    // where pages have places by the call's tokens, every page that a sequence can touch
    // has one of its own, and all are launched
    std::mt19937 rng(1);
    for (int trial = 0; trial < 3000; ++trial) {
        const int shift = 4 + (int)(rng() % 4), P = 1 << shift, B = 1 + (int)(rng() % 40);
        int64_t at = 0, next = 0;
        for (int s = 0; s < B; ++s) {
            const int64_t held = rng() % 300, m = rng() % 3 == 0 ? rng() % 500 : rng() % 4;
            const int64_t pages = m == 0 ? 0 : (held + m - 1) / P - held / P + 1;
            const int64_t first = sffn::first_place((int)at, s, shift);
            EXPECT(first >= next && pages <= sffn::pages_touched(m, P));
            next = first + (pages > 0 ? pages : 1);
            at += m;
        }
        EXPECT(next <= sffn::places_by_tokens(at, B, P));
    }
    // all sizes of the header's ranges are taken or refused, none fails in a launch
    for (int heads : {1, 8, 64, 1000})
        for (int page : {16, 128})
            for (int seqs : {1, 1000, 1 << 20})
                for (int64_t tokens : {(int64_t)1, (int64_t)5000, (int64_t)1 << 22, (int64_t)1 << 28}) {
                    c.kv_heads = heads; c.page = page;
                    b.n_seqs = seqs; b.max_new = INT32_MAX;
                    const sffn_heads_t x{dev(17), (int64_t)heads * 128, 128};
                    const sffn_status_t st = kv_cache_append(&c, &b, &x, &x, SFFN_BF16, tokens, nullptr);
                    const uint64_t k = LAUNCHED();
                    EXPECT(st == SFFN_OK || (st == SFFN_ERR_UNSUPPORTED && k == 0));
                    EXPECT(st != SFFN_OK || k >= (uint64_t)(tokens / page) * heads * 2);
                }

    // ---- attention: row tiles of one prompt's length for each of many sequences -------
    c.kv_heads = 8; c.page = 64;
    b.n_seqs = 1024; b.max_pages = 2048; b.table_stride = 2048; b.max_new = 131072;
    const sffn_heads_t h{dev(18), 4096, 128};
    for (int window : {0, 1000})
        for (int seqs : {1, 64, 1024, 8000}) {
            b.n_seqs = seqs;
            const sffn_status_t st = cache_attention(&c, &b, &h, 32, SFFN_BF16, 131072 + seqs - 1, 0.1f, window, &h,
                                                     nullptr, dev(19), (size_t)-1, nullptr);
            EXPECT(st == SFFN_OK);
            EXPECT(LAUNCHED() >= (uint64_t)131072 * 4 / 256 * 8);
        }

    if (g_failed) {
        std::printf("%d checks failed\n", g_failed);
        return 1;
    }
    std::printf("launch checks passed\n");
    return 0;
}
