// The C entry points and launchers of the norm, the page bookkeeping and the 4-bit cache
// against a faked HIP runtime that records every launch: sizes at the ends of their ranges,
// each launch within HIP's limit (fewer than 2^32 threads in a grid) and all of them
// together enough for the work, workspaces as their sizes say, the propagation of HIP
// errors. Built with the sanitizers and run by tests/test_layer_host_hardening.py.
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <vector>

#include <hip/hip_runtime.h>

#include "attn_launch.hpp"
#include "sparse_ffn_attention.h"
#include "sparse_ffn_norm.h"
#include "sparse_ffn_paging.h"
#include "status.hpp"

alignas(256) unsigned char fake_fatbin[64];

struct Launch {
    uint64_t blocks, threads;
};
static std::vector<Launch> g_launches;
static dim3 g_grid, g_block;
static hipError_t g_status = hipSuccess;
static int g_zeros = 0;

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
hipError_t hipGetLastError() { return g_status; }
const char* hipGetErrorString(hipError_t) { return "injected HIP error"; }
hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) { *v = 256; return hipSuccess; }
}
namespace sffn {
hipError_t launch_zero_f32(float*, int64_t, hipStream_t) { ++g_zeros; return g_status; }
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
template <typename T> static T* at(uintptr_t k) { return static_cast<T*>(dev(k)); }

// Threads of the launches since the last call, each within the limit.
static uint64_t launched(int line) {
    uint64_t sum = 0;
    for (const Launch& l : g_launches) {
        expect(l.blocks >= 1 && l.threads <= 1024 && l.blocks * l.threads < (uint64_t)1 << 32,
               "a grid of fewer than 2^32 threads", line);
        sum += l.blocks * l.threads;
    }
    g_launches.clear();
    return sum;
}
#define LAUNCHED() launched(__LINE__)

static void norms() {
    const sffn_rows_t x{dev(1), 1 << 20}, y{dev(2), 1 << 20};
    for (int dtype : {SFFN_F32, SFFN_BF16})
        for (int out : {SFFN_NORM_SAME, SFFN_NORM_INT8, SFFN_NORM_E4M3})
            for (int d : {1, 7, 512, 513, 1024, 2049, 4096, 8192, 14336, 16384, 32768, 32769, 1 << 20})
                for (int64_t T : {(int64_t)1, (int64_t)5, (int64_t)4096, (int64_t)1 << 24, (int64_t)1 << 30}) {
                    sffn_norm_config_t c{};
                    c.d = d;
                    c.eps = 1e-6f;
                    std::memcpy(&c.dtype, &dtype, sizeof dtype);
                    std::memcpy(&c.out, &out, sizeof out);
                    EXPECT_STATUS(add_rms_norm(&c, T, &x, &x, dev(3), &y, at<float>(4), &x, nullptr), SFFN_OK);
                    EXPECT(LAUNCHED() >= (uint64_t)T * 64);
                    const size_t need = add_rms_norm_backward_workspace_size(&c, T);
                    EXPECT(need >= (size_t)d * 4 && need <= (size_t)256 * d * 4);
                    EXPECT_STATUS(add_rms_norm_backward(&c, T, &x, &x, &x, dev(3), &y, at<float>(4), dev(5), need, nullptr), SFFN_OK);
                    EXPECT(LAUNCHED() >= 512);
                    EXPECT_STATUS(add_rms_norm_backward(&c, T, &x, &x, nullptr, nullptr, &y, nullptr, nullptr, 0, nullptr), SFFN_OK);
                    EXPECT(LAUNCHED() >= 512);
                }
    sffn_norm_config_t c{};
    c.d = 64;
    c.dtype = SFFN_BF16;
    c.eps = 1e-6f;
    for (int64_t T : {((int64_t)1 << 30) + 1, INT64_MAX}) {
        EXPECT_STATUS(add_rms_norm(&c, T, &x, &x, nullptr, &y, nullptr, nullptr, nullptr), SFFN_ERR_UNSUPPORTED);
        EXPECT(add_rms_norm_backward_workspace_size(&c, T) == 0);
    }
    for (int bad : {INT_MIN, -1, 3, INT_MAX}) {
        sffn_norm_config_t b = c;
        std::memcpy(&b.dtype, &bad, sizeof bad);
        EXPECT_STATUS(add_rms_norm(&b, 4, &x, nullptr, nullptr, &y, nullptr, nullptr, nullptr), SFFN_ERR_INVALID_ARG);
        b = c;
        std::memcpy(&b.out, &bad, sizeof bad);
        EXPECT_STATUS(add_rms_norm(&b, 4, &x, nullptr, nullptr, &y, nullptr, nullptr, nullptr), SFFN_ERR_INVALID_ARG);
    }
    const int zeros = g_zeros;
    EXPECT_STATUS(add_rms_norm_backward(&c, 0, nullptr, nullptr, nullptr, nullptr, nullptr, at<float>(4), nullptr, 0, nullptr), SFFN_OK);
    EXPECT(g_zeros == zeros + 1 && LAUNCHED() == 0);
}

static void pages() {
    sffn_page_pool_t p{};
    p.block_table = at<int32_t>(1);
    p.free_pages = at<int32_t>(2);
    sffn_kv_batch_t b{};
    b.block_table = at<int32_t>(1);
    b.kv_lens = at<int32_t>(3);
    b.cu = at<int32_t>(4);
    for (int page : {16, 128})
        for (int seqs : {0, 1, 256, 257, 5000, 1 << 24})
            for (int max_pages : {1, 512, (1 << 30) / page})
                for (int64_t T : {(int64_t)0, (int64_t)1, (int64_t)1024, (int64_t)1025, (int64_t)4097, (int64_t)1 << 28}) {
                    p.n_pages = INT32_MAX; p.n_seqs = seqs; p.max_pages = max_pages; p.table_stride = max_pages; p.page = page;
                    EXPECT_STATUS(page_plan(&p, at<int32_t>(5), nullptr, at<int32_t>(6), at<int32_t>(7), T, at<int32_t>(5),
                                            at<int32_t>(7), at<int32_t>(8), at<int32_t>(9), at<int64_t>(10), nullptr), SFFN_OK);
                    EXPECT(LAUNCHED() >= (T > 2048 ? (uint64_t)T : 256));
                    b.n_seqs = seqs; b.max_pages = max_pages; b.table_stride = max_pages; b.max_new = INT32_MAX;
                    EXPECT_STATUS(cache_slots(&b, INT32_MAX, page, T, at<int32_t>(9), at<int64_t>(10), nullptr), SFFN_OK);
                    EXPECT(LAUNCHED() >= (uint64_t)T);
                }
}

static void caches() {
    sffn_kv_cache4_t c{};
    c.keys = at<uint8_t>(10); c.values = at<uint8_t>(11); c.k_exp = at<uint8_t>(12); c.v_scale = at<float>(13);
    c.n_pages = INT32_MAX; c.kv_heads = 8; c.page = 64; c.head_dim = 128;
    sffn_kv_batch_t b{};
    b.block_table = at<int32_t>(14); b.kv_lens = at<int32_t>(15); b.cu = at<int32_t>(16);
    b.n_seqs = 4; b.max_pages = 1000; b.table_stride = 1000; b.max_new = 300; b.max_kv = 60000;
    const int64_t* slots = at<int64_t>(20);
    for (int dim : {64, 128, 256})
        for (int dtype : {SFFN_F32, SFFN_BF16})
            for (int64_t T : {(int64_t)1, (int64_t)4095, (int64_t)1 << 22, (int64_t)1 << 27}) {
                c.head_dim = dim;
                sffn_dtype_t dt;
                std::memcpy(&dt, &dtype, sizeof dt);
                const sffn_heads_t kv{dev(17), 8 * dim, dim};
                EXPECT_STATUS(kv_cache4_append(&c, nullptr, slots, &kv, &kv, dt, T, nullptr), SFFN_OK);
                EXPECT(LAUNCHED() >= (uint64_t)T * 8 * dim / 8);
                EXPECT_STATUS(kv_cache4_append(&c, &b, nullptr, &kv, &kv, dt, T, nullptr), SFFN_OK);
                EXPECT(LAUNCHED() >= (uint64_t)T * 8 * dim / 8);
                EXPECT_STATUS(kv_cache4_read(&c, &b, &kv, &kv, dt, T, nullptr), SFFN_OK);
                EXPECT(LAUNCHED() >= (uint64_t)T * 8 * dim / 8);
            }
    c.head_dim = 128;
    const sffn_heads_t kv{dev(17), 1024, 128};
    for (int64_t T : {(int64_t)-1, ((int64_t)1 << 28) + 1, (int64_t)1 << 31, INT64_MAX})
        EXPECT(kv_cache4_append(&c, nullptr, slots, &kv, &kv, SFFN_BF16, T, nullptr) != SFFN_OK);
    EXPECT_STATUS(kv_cache4_append(&c, nullptr, nullptr, &kv, &kv, SFFN_BF16, 4, nullptr), SFFN_ERR_INVALID_ARG);
    EXPECT_STATUS(kv_cache4_append(&c, &b, reinterpret_cast<const int64_t*>(4), &kv, &kv, SFFN_BF16, 4, nullptr), SFFN_ERR_INVALID_ARG);
    EXPECT_STATUS(kv_cache4_append(&c, nullptr, slots, nullptr, nullptr, SFFN_BF16, 0, nullptr), SFFN_OK);
    EXPECT(LAUNCHED() == 0);

    // plans over the whole range stay within a grid, and their workspace is what the size says
    for (int dim : {64, 128, 256})
        for (int heads : {8, 32, 128})
            for (int seqs : {1, 4, 1000})
                for (int new_tokens : {0, 1, 2, 5, 17, 300, 1 << 20, INT32_MAX})
                    for (int kv_len : {0, 1, 513, 60000, INT32_MAX})
                        for (int window : {0, 700, INT32_MAX})
                            for (int64_t T : {(int64_t)1, (int64_t)4096, (int64_t)1 << 20}) {
                                sffn_kv_batch_t x = b;
                                c.head_dim = dim;
                                x.n_seqs = seqs; x.max_new = new_tokens; x.max_kv = kv_len;
                                const size_t ws = cache4_attention_workspace_size(&c, &x, heads, SFFN_BF16, window, T);
                                EXPECT(ws <= (size_t)256 << 20);
                                const sffn_heads_t h{dev(18), (int64_t)heads * dim, dim};
                                const sffn_status_t st = cache4_attention(&c, &x, &h, heads, SFFN_BF16, T, 0.1f, window, &h,
                                                                          nullptr, dev(19), ws, nullptr);
                                const uint64_t n = LAUNCHED();
                                EXPECT(st == SFFN_OK || (st == SFFN_ERR_UNSUPPORTED && n == 0));
                                EXPECT(st != SFFN_OK || new_tokens == 0 || n >= 256);
                                if (ws > 0)
                                    EXPECT_STATUS(cache4_attention(&c, &x, &h, heads, SFFN_BF16, T, 0.1f, window, &h, nullptr,
                                                                   dev(19), ws - 1, nullptr), SFFN_ERR_WORKSPACE);
                            }
    c.head_dim = 128;
    // what the kernels count in 31 bits: steps and the cost of every unit
    sffn_kv_batch_t x = b;
    for (int seqs : {100000, 1 << 22, INT32_MAX}) {
        x.n_seqs = seqs; x.max_pages = 1 << 18; x.table_stride = 1 << 18;
        const sffn_heads_t h{dev(18), 4096, 128};
        EXPECT_STATUS(cache4_attention(&c, &x, &h, 32, SFFN_BF16, 4096, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr),
                      SFFN_ERR_UNSUPPORTED);
    }
    EXPECT(LAUNCHED() == 0);
}

static void errors() {
    g_status = hipErrorLaunchFailure;
    sffn_norm_config_t n{};
    n.d = 64; n.dtype = SFFN_BF16; n.eps = 1e-6f;
    const sffn_rows_t x{dev(1), 64}, y{dev(2), 64};
    EXPECT_STATUS(add_rms_norm(&n, 4, &x, nullptr, nullptr, &y, nullptr, nullptr, nullptr), SFFN_ERR_HIP);
    EXPECT(std::strstr(sffn::last_error, "add_rms_norm") != nullptr);
    EXPECT_STATUS(add_rms_norm_backward(&n, 4, &x, &x, nullptr, nullptr, &y, nullptr, nullptr, 0, nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(add_rms_norm_backward(&n, 0, &x, &x, nullptr, nullptr, &y, at<float>(3), nullptr, 0, nullptr), SFFN_ERR_HIP);
    sffn_page_pool_t p{at<int32_t>(1), 5, at<int32_t>(2), 100, 3, 5, 16};
    EXPECT_STATUS(page_plan(&p, at<int32_t>(5), nullptr, at<int32_t>(6), at<int32_t>(7), 9, at<int32_t>(5), at<int32_t>(7),
                            at<int32_t>(8), at<int32_t>(9), at<int64_t>(10), nullptr), SFFN_ERR_HIP);
    EXPECT(std::strstr(sffn::last_error, "page_plan") != nullptr);
    sffn_kv_cache4_t c{at<uint8_t>(10), at<uint8_t>(11), at<uint8_t>(12), at<float>(13), 100, 8, 64, 128};
    sffn_kv_batch_t b{at<int32_t>(14), 10, at<int32_t>(15), at<int32_t>(16), 4, 10, 300, 600};
    const sffn_heads_t kv{dev(17), 1024, 128}, h{dev(18), 4096, 128};
    EXPECT_STATUS(cache_slots(&b, 100, 64, 9, at<int32_t>(9), at<int64_t>(10), nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(kv_cache4_append(&c, &b, nullptr, &kv, &kv, SFFN_BF16, 9, nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(kv_cache4_read(&c, &b, &kv, &kv, SFFN_BF16, 9, nullptr), SFFN_ERR_HIP);
    EXPECT_STATUS(cache4_attention(&c, &b, &h, 32, SFFN_BF16, 9, 0.1f, 0, &h, nullptr, dev(19), (size_t)-1, nullptr), SFFN_ERR_HIP);
    EXPECT(std::strstr(sffn::last_error, "cache4_attention") != nullptr);
}

int main() {
    norms();
    pages();
    caches();
    errors();
    if (g_failed) {
        std::printf("%d checks failed\n", g_failed);
        return 1;
    }
    std::printf("layer checks passed\n");
    return 0;
}
