// softmax_inst.hip -- instantiates the softmax kernels for one operand type and width, given as
// MIPS_CT (MIPS_F32 or MIPS_BF16) and MIPS_D by the build; one object per pair keeps each
// compilation small and lets them run in parallel.
#include "softmax.h"
#include "softmax_grad.h"

#if !defined(MIPS_CT) || !defined(MIPS_D)
#error "MIPS_CT and MIPS_D must be defined"
#endif

namespace mips {
template int launch_stats<MIPS_CT, MIPS_D>(int, bool, const StatsArgs&, int, hipStream_t);
#if MIPS_D >= 32
template int launch_grad<MIPS_CT, MIPS_D>(bool, bool, const GradArgs&, hipStream_t);
#endif
}  // namespace mips
