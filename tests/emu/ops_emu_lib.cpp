// Host-emulated build of the operators around the scan (TEST INFRASTRUCTURE): the C-ABI
// source is compiled unchanged against the emulated device headers next to this file.
#include "../../complex_chunkwise_ssd_amd/csrc/ssd_ops_api.hip"

extern "C" void emu_set_shuffle_seed(unsigned long long seed) { emu::g_shuffle = seed; }
