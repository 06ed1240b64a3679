// Bounds and races of the operators around the scan under a sanitizer on the host (TEST
// INFRASTRUCTURE). Every buffer is an exact-size heap allocation, so that AddressSanitizer ends the run
// at any read or write past a tensor or a shared-memory array; under ThreadSanitizer, accesses of
// two waves that no barrier orders are reported. Values are checked elsewhere.
#include "ops_emu_lib.cpp"

#include <math.h>
#include <stdio.h>
#include <stdlib.h>
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
    uint8_t *u() const { return (uint8_t *)at; }
};
struct Values : Buffer {  // uniform in +-2
    Values(size_t n, int dtype) : Buffer(n * (size_t)elem_size(dtype))
    {
        for (size_t i = 0; i < n; ++i) {
            const float v = 4.f * uniform01() - 2.f;
            if (dtype == SSD_F32)
                f()[i] = v;
            else
                ((uint16_t *)at)[i] = (uint16_t)(f2u(v) >> 16);
        }
    }
};
struct Bytes : Buffer {  // e4m3 without NaN
    explicit Bytes(size_t n) : Buffer(n)
    {
        for (size_t i = 0; i < n; ++i)
            u()[i] = (uint8_t)((unsigned)(uniform01() * 256.f) & 0xf7u);
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

void gated(int64_t B, int64_t T, int64_t C, int dtype, const std::vector<int32_t> &lengths)
{
    printf("gated %d x %d x %d type %d\n", (int)B, (int)T, (int)C, dtype);
    const size_t n = (size_t)(B * T * C), bc = (size_t)(B * C), e = (size_t)elem_size(dtype);
    const size_t chunks = (size_t)((T + SSD_GATED_CHUNK - 1) / SSD_GATED_CHUNK);
    Values x(n, dtype), gi(n, dtype), gr(n, dtype), gh(n, dtype), lam((size_t)C, SSD_F32), init(bc, SSD_F32);
    Buffer h(n * e), states((size_t)B * chunks * (size_t)C * 4), gx(n * e), ggi(n * e), ggr(n * e), glam((size_t)C * 4),
        ginit(bc * 4), len(lengths.size() * 4);
    memcpy(len.at, lengths.data(), lengths.size() * 4);
    const int32_t *L = lengths.empty() ? nullptr : (const int32_t *)len.at;
    const size_t need = ssd_gated_scan_workspace_bytes(B, T, C, dtype);
    Workspace w(need);
    // the state in place
    expect_ok(ssd_gated_scan(x, C, gi, C, gr, C, lam.f(), 8.f, dtype, B, T, C, init.f(), L, h, init.f(), states.f(), w.at,
                             need, nullptr), "gated");
    const size_t more = ssd_gated_scan_backward_workspace_bytes(B, T, C, dtype);
    Workspace v(more);
    expect_ok(ssd_gated_scan_backward(x, C, gi, C, gr, C, lam.f(), 8.f, dtype, B, T, C, states.f(), L, gh, init.f(), gx, ggi,
                                      ggr, glam.f(), ginit.f(), v.at, more, nullptr), "gated backward");
}

void norm(int64_t rows, int64_t F, int dtype)
{
    printf("norm %d x %d type %d\n", (int)rows, (int)F, dtype);
    const size_t n = (size_t)(rows * F), e = (size_t)elem_size(dtype), kb = (size_t)((F + 127) / 128);
    Values x(n, dtype), res(n, dtype), gy(n, dtype), w((size_t)F, SSD_F32);
    Buffer y(n * e), q(n), scale(kb * (size_t)rows * 4), rstd((size_t)rows * 4), gx(n * e), gw((size_t)F * 4);
    // the residual in place
    expect_ok(ssd_rms_norm(x, F, res, F, w.f(), dtype, rows, F, 1e-6f, y, res, q.u(), scale.f(), rstd.f(), nullptr), "norm");
    const size_t need = ssd_rms_norm_backward_workspace_bytes(rows, F);
    Workspace v(need);
    expect_ok(ssd_rms_norm_backward(res, F, w.f(), rstd.f(), gy, F, x, F, dtype, rows, F, gx, gw.f(), v.at, need, nullptr),
              "norm backward");
}

void quantise(int64_t rows, int64_t cols, int dtype)
{
    printf("quantise %d x %d type %d\n", (int)rows, (int)cols, dtype);
    Values x((size_t)(rows * cols), dtype);
    for (int block_rows = 1; block_rows <= 128; block_rows += 127)
        for (int turn = 0; turn < 2; ++turn) {
            const int64_t R = turn ? cols : rows, K = turn ? rows : cols;
            Buffer q((size_t)(R * K)), scale((size_t)((K + 127) / 128 * (block_rows == 1 ? R : (R + 127) / 128)) * 4);
            expect_ok(ssd_fp8_quantise(x, cols, dtype, rows, cols, block_rows, turn, q.u(), K, scale.f(), nullptr), "quantise");
        }
}

void matmul(int64_t M, int64_t N, int64_t K, int out_dtype, bool large_tiles = false)
{
    printf("matmul %d x %d x %d out %d%s\n", (int)M, (int)N, (int)K, out_dtype, large_tiles ? ", tiles of 256 x 256" : "");
    const int64_t kb = (K + 127) / 128;
    for (int block_rows = 1; block_rows <= 128; block_rows += 127) {
        Bytes a((size_t)(M * K)), b((size_t)(N * K));
        Values sa((size_t)(kb * M), SSD_F32), sb((size_t)(kb * (block_rows == 1 ? N : (N + 127) / 128)), SSD_F32);
        Buffer out((size_t)(M * N * elem_size(out_dtype)));
        if (large_tiles) {
            Buffer part((size_t)(2 * M * N) * 4);
            expect_ok(emu_fp8_big(a.u(), sa.f(), b.u(), sb.f(), (int)M, (int)N, (int)K, block_rows, 2, out, part.f()), "matmul");
            continue;
        }
        const int on16 = K % 16 == 0;  // heap blocks start on 16 bytes
        const size_t need = ssd_fp8_matmul_workspace_bytes(M, N, K, block_rows, out_dtype, on16);
        Workspace w(need);
        expect_ok(ssd_fp8_matmul(a.u(), K, sa.f(), b.u(), K, sb.f(), M, N, K, block_rows, out_dtype, out, N, w.at, need, nullptr),
                  "matmul");
    }
}

}  // namespace

int main()
{
    for (int t = 0; t < 2; ++t) {
        gated(1, 1, 3, t, {});
        gated(2, 9, 65, t, {9, 3});
        gated(1, 700, 66, t, {INT32_MIN});
        gated(3, 200, 130, t, {0, 200, 77});
    }
    gated(1, 1100, 132, SSD_BF16, {1050});
    norm(1, 1, SSD_F32);
    norm(18, 65, SSD_BF16);
    norm(5, 600, SSD_F32);
    norm(6, 1030, SSD_BF16);
    norm(2, 8193, SSD_F32);
    quantise(130, 259, SSD_BF16);
    quantise(5, 17, SSD_F32);
    for (int t = 0; t < 2; ++t) {
        matmul(3, 20, 130, t);
        matmul(20, 33, 1300, t);
        matmul(70, 90, 400, t);
        matmul(66, 40, 2999, t);
    }
    matmul(257, 130, 400, SSD_BF16, true);
    if (!failed)
        printf("OK\n");
    return failed;
}
