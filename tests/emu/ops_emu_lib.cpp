// Host-emulated build of the operators around the scan (TEST INFRASTRUCTURE): the C-ABI
// source is compiled unchanged against the emulated device headers next to this file.
#include "../../complex_chunkwise_ssd_amd/csrc/ssd_ops_api.hip"

extern "C" void emu_set_shuffle_seed(unsigned long long seed) { emu::g_shuffle = seed; }

// The form that a call takes: what the tests of the forms are checked against.
extern "C" void emu_fp8_form(int64_t M, int64_t N, int64_t K, int out_dtype, int aligned_rows, int64_t *form)
{
    const Fp8Plan p = fp8_plan(M, N, K, out_dtype, aligned_rows != 0);
    form[0] = p.few;
    form[1] = p.mb;
    form[2] = p.waves;
    form[3] = p.splits;
    form[4] = (int64_t)p.tiles_m * p.tiles_n;
}
extern "C" void emu_gated_form(int64_t batch, int64_t T, int64_t C, int dtype, int backward, int64_t *form)
{
    const GatedPlan p = gated_plan(batch, T, C, dtype, backward != 0);
    form[0] = p.ch;
    form[1] = p.segments;
    form[2] = p.walk;
}

// The large form of the product with tiles of 256 x 256, which a plan takes for larger calls than the
// emulator's.
extern "C" int emu_fp8_big(const uint8_t *a, const float *sa, const uint8_t *b, const float *sb, int M, int N, int K,
                           int b_block_rows, int splits, void *out, float *part)
{
    ssd::Fp8Params p{};
    p.a = a;
    p.b = b;
    p.sa = sa;
    p.sb = sb;
    p.out = out;
    p.part = part;
    p.a_stride = p.b_stride = K;
    p.out_stride = N;
    p.M = M;
    p.N = N;
    p.K = K;
    Fp8Plan plan{};
    plan.mb = 8;
    p.tiles_m = plan.tiles_m = (M + 255) / 256;
    p.tiles_n = plan.tiles_n = (N + 255) / 256;
    const int kb = (K + 127) / 128;
    p.split_blocks = plan.split_blocks = (kb + splits - 1) / splits;
    p.splits = plan.splits = (kb + p.split_blocks - 1) / p.split_blocks;
    return b_block_rows == 1 ? launch_fp8<true, ssd::kBF16>(p, plan, true, nullptr, nullptr)
                             : launch_fp8<false, ssd::kBF16>(p, plan, true, nullptr, nullptr);
}
