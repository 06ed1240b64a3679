// Alignment of what the gated delta rule reads and writes (TEST INFRASTRUCTURE), for -fsanitize=alignment on the host: in shared
// memory, and in tensors that lie `argv[1]` elements past a boundary of 256 bytes (the workspace is always on one). Ends
// with a number made of all results, the same for every such place. With "limits", for -fsanitize=signed-integer-overflow,
// the arithmetic on sizes.
#include "delta_emu_lib.cpp"

#include <stddef.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

namespace {

size_t off = 0;
uint64_t sum = 0;

struct Tensor {
    char *base, *at;
    size_t bytes;
    Tensor(size_t n, size_t e) : base((char *)aligned_alloc(256, (n * e + off * e + 511) & ~(size_t)255)), at(base + off * e), bytes(n * e)
    {
        memset(at, 0, bytes);
    }
    Tensor(const Tensor &) = delete;
    ~Tensor() { free(base); }
    operator void *() const { return at; }
    float *f() const { return (float *)at; }
    void add() const
    {
        for (size_t i = 0; i < bytes; ++i)
            sum = sum * 0x100000001b3ULL + (unsigned char)at[i];
    }
};
struct Values : Tensor {  // uniform in low .. high
    Values(size_t n, int dtype, float low, float high) : Tensor(n, dtype == SSD_F32 ? 4 : 2)
    {
        static unsigned seed = 1;
        for (size_t i = 0; i < n; ++i) {
            seed = seed * 1664525u + 1013904223u;
            const float v = low + (high - low) * ((float)(seed >> 8) * (1.f / 16777216.f));
            uint32_t u;
            memcpy(&u, &v, 4);
            if (dtype == SSD_F32)
                memcpy(at + 4 * i, &u, 4);
            else
                ((uint16_t *)at)[i] = (uint16_t)(u >> 16);
        }
    }
};

// One head; `rows` - 1 of the rows are empty.
bool delta(int rows, int T, int Dk, int Dv, int dtype)
{
    printf("delta %d x %d, %d x %d, type %d\n", rows, T, Dk, Dv, dtype);
    fflush(stdout);
    const size_t e = dtype == SSD_F32 ? 4 : 2, nk = (size_t)rows * T * Dk, nv = (size_t)rows * T * Dv, ng = (size_t)rows * T;
    const size_t ns = (size_t)rows * Dk * Dv, chunks = (size_t)((T + 63) / 64);
    const float unit = 1.f / (float)Dk;
    Values q(nk, dtype, -1.f, 1.f), k(nk, dtype, -unit, unit), v(nv, dtype, -1.f, 1.f), go(nv, dtype, -1.f, 1.f);
    Values g(ng, SSD_F32, -1.f, 0.f), beta(ng, SSD_F32, 0.f, 1.f), state(ns, SSD_F32, -1.f, 1.f);
    Tensor o(nv, e), fin(ns, 4), states(ns * chunks, 4), gq(nk, e), gk(nk, e), gv(nv, e), gg(ng, 4), gb(ng, 4), g0(ns, 4);
    Tensor len((size_t)rows, 4);
    ((int32_t *)len.at)[rows / 2] = T;
    const size_t n0 = ssd_gated_delta_workspace_bytes(rows, T, 1, 1, Dk, Dv, dtype);
    const size_t n1 = ssd_gated_delta_backward_workspace_bytes(rows, T, 1, 1, Dk, Dv, dtype);
    void *ws = aligned_alloc(256, ((n0 > n1 ? n0 : n1) + 511) & ~(size_t)255);
    const int st = ssd_gated_delta(q, Dk, k, Dk, v, Dv, g.f(), beta.f(), 0.5f, dtype, rows, T, 1, 1, Dk, Dv, state.f(),
                                   (int32_t *)len.at, o, fin.f(), states.f(), ws, n0, nullptr);
    const int bwd = ssd_gated_delta_backward(q, Dk, k, Dk, v, Dv, g.f(), beta.f(), 0.5f, dtype, rows, T, 1, 1, Dk, Dv, states.f(),
                                             (int32_t *)len.at, go, state.f(), gq, gk, gv, gg.f(), gb.f(), g0.f(), ws, n1, nullptr);
    free(ws);
    for (const Tensor *t : {&o, &fin, &states, &gq, &gk, &gv, &gg, &gb, &g0})
        t->add();
    return st == SSD_OK && bwd == SSD_OK;
}

// What is read in vectors of 16 bytes through a structure in shared memory starts on such a boundary (the sanitizer does not
// see these: the compiler knows where a member lies and loads it as the place allows).
bool on16(size_t at, const char *what)
{
    if (at % 16 != 0)
        printf("%s: %d past a boundary of 16 bytes\n", what, (int)(at % 16));
    return at % 16 == 0;
}
bool gates_placed()
{
    typedef ssd::DeltaGates G;
    return on16(sizeof(G), "gates, the second of two") && on16(alignof(G), "gates") && on16(offsetof(G, since), "since") &&
           on16(offsetof(G, left), "left") && on16(offsetof(G, beta), "beta");
}
template <int T, int KP, bool MANY>
bool grad_placed()
{
    typedef ssd::GradLds<T, KP, MANY> L;
    return on16(offsetof(L, own_tri), "triangle") && on16(offsetof(L, k), "keys") && on16(offsetof(L, own_kt), "keys by features") &&
           on16(offsetof(L, gates), "gates of the gradients") && on16(alignof(L), "gradients");
}
template <int T>
bool grads_placed()
{
    return grad_placed<T, 2, false>() && grad_placed<T, 2, true>() && grad_placed<T, 4, false>() && grad_placed<T, 4, true>();
}

}  // namespace

// Sizes past the limits whose product passes 2^63: no workspace, whatever it wraps to.
bool limits()
{
    const int64_t M = 1 << 24, T = 1 << 30, H = 1 << 16;
    bool ok = true;
    for (int64_t B : {M, M - 1, M / 2 + 5})
        for (int64_t t : {T, T - 64, T / 2})
            ok = ok && ssd_gated_delta_workspace_bytes(B, t, 1, H, 16, 32, SSD_BF16) == 0 &&
                 ssd_gated_delta_backward_workspace_bytes(B, t, 1, H, 16, 32, SSD_BF16) == 0;
    printf(ok ? "OK \n" : "a workspace\n");
    return ok;
}

int main(int, char **argv)
{
    if (strcmp(argv[1], "limits") == 0)
        return !limits();
    off = (size_t)atoi(argv[1]);
    bool ok = gates_placed() && grads_placed<ssd::kF32>() && grads_placed<ssd::kBF16>();
    if (!ok)
        return 1;
    for (int dtype : {SSD_F32, SSD_BF16}) {
        ok = delta(2, 5, 20, 24, dtype) && ok;       // token by token
        ok = delta(1, 140, 32, 40, dtype) && ok;     // few heads, and columns in one piece and in two
        ok = delta(1, 140, 72, 68, dtype) && ok;
        ok = delta(193, 140, 32, 40, dtype) && ok;   // many
        ok = delta(193, 140, 72, 36, dtype) && ok;
        ok = delta(97, 140, 72, 68, dtype) && ok;
    }
    printf(ok ? "OK %016llx\n" : "a call was refused\n", (unsigned long long)sum);
    return !ok;
}
