// Bounds and races of the gated delta rule and of the norms around a block under a sanitizer on the host (TEST
// INFRASTRUCTURE), as ops_emu_main.cpp: every buffer is an exact-size heap allocation. Values are checked elsewhere.
#include "delta_emu_lib.cpp"
#include "../../complex_chunkwise_ssd_amd/csrc/ssd_block_api.hip"

#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <vector>

namespace {

unsigned seed = 1;
float uniform01()
{
    seed = seed * 1664525u + 1013904223u;
    return (float)(seed >> 8) * (1.f / 16777216.f);
}

struct Buffer {
    char *at;
    explicit Buffer(size_t bytes) : at((char *)malloc(bytes + (bytes == 0))) {}
    Buffer(const Buffer &) = delete;
    ~Buffer() { free(at); }
    operator void *() const { return at; }
    float *f() const { return (float *)at; }
};
struct Values : Buffer {  // uniform in low .. high
    Values(size_t n, int dtype, float low, float high) : Buffer(n * (dtype == SSD_F32 ? 4 : 2))
    {
        for (size_t i = 0; i < n; ++i) {
            const float v = low + (high - low) * uniform01();
            uint32_t u;
            memcpy(&u, &v, 4);
            if (dtype == SSD_F32)
                f()[i] = v;
            else
                ((uint16_t *)at)[i] = (uint16_t)(u >> 16);
        }
    }
};
struct Workspace {
    void *at;
    explicit Workspace(size_t n) : at(n ? aligned_alloc(256, (n + 255) & ~(size_t)255) : nullptr) {}
    ~Workspace() { free(at); }
};

int failed = 0;
void expect_ok(int status, const char *what)
{
    if (status != SSD_OK) {
        printf("%s: status %d\n", what, status);
        failed = 1;
    }
}

void delta(int64_t B, int64_t T, int64_t Hk, int64_t Hv, int64_t Dk, int64_t Dv, int dtype, const std::vector<int32_t> &lengths)
{
    printf("delta %d x %d, heads %d %d of %d %d, type %d\n", (int)B, (int)T, (int)Hk, (int)Hv, (int)Dk, (int)Dv, dtype);
    const size_t e = dtype == SSD_F32 ? 4 : 2, nk = (size_t)(B * T * Hk * Dk), nv = (size_t)(B * T * Hv * Dv);
    const size_t ng = (size_t)(B * T * Hv), ns = (size_t)(B * Hv * Dk * Dv), chunks = (size_t)((T + 63) / 64);
    const float unit = 1.f / (float)Dk;
    Values q(nk, dtype, -1.f, 1.f), k(nk, dtype, -unit, unit), v(nv, dtype, -1.f, 1.f), go(nv, dtype, -1.f, 1.f);
    Values g(ng, SSD_F32, -1.f, 0.f), beta(ng, SSD_F32, 0.f, 1.f), state(ns, SSD_F32, -1.f, 1.f);
    Buffer o(nv * e), states(ns * chunks * 4), gq(nk * e), gk(nk * e), gv(nv * e), gg(ng * 4), gb(ng * 4), g0(ns * 4);
    Buffer len(lengths.size() * 4);
    memcpy(len.at, lengths.data(), lengths.size() * 4);
    const int32_t *L = lengths.empty() ? nullptr : (const int32_t *)len.at;
    const size_t need = ssd_gated_delta_workspace_bytes(B, T, Hk, Hv, Dk, Dv, dtype);
    Workspace w(need);
    // the state in place
    expect_ok(ssd_gated_delta(q, Hk * Dk, k, Hk * Dk, v, Hv * Dv, g.f(), beta.f(), 0.5f, dtype, B, T, Hk, Hv, Dk, Dv, state.f(),
                              L, o, state.f(), states.f(), w.at, need, nullptr), "delta");
    const size_t more = ssd_gated_delta_backward_workspace_bytes(B, T, Hk, Hv, Dk, Dv, dtype);
    Workspace x(more);
    expect_ok(ssd_gated_delta_backward(q, Hk * Dk, k, Hk * Dk, v, Hv * Dv, g.f(), beta.f(), 0.5f, dtype, B, T, Hk, Hv, Dk, Dv,
                                       states.f(), L, go, state.f(), gq, gk, gv, gg.f(), gb.f(), g0.f(), x.at, more, nullptr),
              "delta backward");
}

std::vector<int32_t> mostly_padding(int rows, int longest)
{
    std::vector<int32_t> n(rows, 0);
    n[rows / 2] = longest;
    n[rows - 1] = longest / 2;
    return n;
}

void norms(int64_t rows, int64_t F, int64_t D, int dtype)
{
    printf("norms %d x %d by %d, type %d\n", (int)rows, (int)F, (int)D, dtype);
    const size_t n = (size_t)(rows * F), e = dtype == SSD_F32 ? 4 : 2, r = (size_t)rows, f = (size_t)F;
    Values x(n, dtype, -2.f, 2.f), z(n, dtype, -2.f, 2.f), gy(n, dtype, -2.f, 2.f), w1(f, SSD_F32, 0.5f, 1.5f), w2(f, SSD_F32, 0.5f, 1.5f);
    Buffer y(n * e), q(n), scale((f + 127) / 128 * r * 4), rstd(n / (size_t)D * 4), r1(r * 4), r2(r * 4), gx(n * e), gz(n * e);
    Buffer g1(f * 4), g2(f * 4);
    expect_ok(ssd_gated_norm(x, F, z, F, w1.f(), dtype, rows, F, D, 1e-6f, y, (uint8_t *)q.at, scale.f(), rstd.f(), nullptr), "gated");
    size_t need = ssd_gated_norm_backward_workspace_bytes(rows, F, D);
    Workspace a(need);
    expect_ok(ssd_gated_norm_backward(x, F, z, F, w1.f(), rstd.f(), gy, F, dtype, rows, F, D, gx, gz, g1.f(), a.at, need, nullptr),
              "gated backward");
    // the residual stream in place
    expect_ok(ssd_block_norm(x, F, z, F, w1.f(), w2.f(), 0.5f, dtype, rows, F, 1e-6f, y, z, (uint8_t *)q.at, scale.f(), r1.f(),
                             r2.f(), nullptr), "block");
    need = ssd_block_norm_backward_workspace_bytes(rows, F);
    Workspace b(need);
    expect_ok(ssd_block_norm_backward(x, F, z, F, w1.f(), w2.f(), r1.f(), r2.f(), 0.5f, gy, F, gy, F, dtype, rows, F, gx, gz, g1.f(),
                                      g2.f(), b.at, need, nullptr), "block backward");
}

}  // namespace

int main()
{
    for (int dtype : {SSD_F32, SSD_BF16}) {
        delta(2, 5, 1, 2, 70, 66, dtype, {5, 0});                // token by token
        delta(2, 140, 1, 2, 33, 20, dtype, {140, 70});           // few heads, two spans of features
        delta(1, 200, 1, 1, 72, 18, dtype, {});                  // four, one of them empty
        // many heads, 64 and 128 columns to a workgroup, and more workgroups of 16 columns than compute units:
        // most rows are padding and cost nothing
        if (dtype == SSD_BF16)
            delta(97, 200, 1, 2, 8, 20, dtype, mostly_padding(97, 200));
        else
            delta(65, 200, 1, 1, 66, 70, dtype, mostly_padding(65, 200));
        delta(97, 200, 1, 1, 66, 66, dtype, mostly_padding(97, 200));
        for (int64_t F : {40, 640, 1400, 2100})
            norms(F == 40 ? 35 : 5, F, F / 4, dtype);
        norms(9, 1024, 64, dtype);
    }
    if (failed)
        return 1;
    printf("OK\n");
    return 0;
}
