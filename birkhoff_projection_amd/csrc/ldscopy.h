// Copies of 16 (or 4) bytes per lane from global memory straight to LDS: from
// a wave-uniform base plus a lane offset to a wave-uniform LDS address (in m0)
// plus 16 (4) bytes per lane.  They are written as assembly because the
// compiler, which cannot tell a stage's buffers apart, would wait for all
// copies before every LDS read.  They have no register result; the wait is the
// vmcnt before the barrier that hands the buffer over.
#pragma once

#include "devmath.h"

namespace mhc {

MHC_DEV void copy16_to_lds(const void* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "m0", "memory");
}

MHC_DEV void copy4_to_lds(const void* base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :: "s"(lds), "v"(off), "s"(base) : "m0", "memory");
}

}  // namespace mhc
