// Host helpers of the calls over sequences (attention, rotary positions, the
// residual step), defined in fpstok_attention_api.cpp.  Not installed; not part
// of the ABI.
#pragma once

#include "fpstok_attention.h"
#include "fpstok_host.h"

namespace fpstok {

inline int elem_bytes(int dtype) { return dtype == FPSTOK_F32 ? 4 : 2; }
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

fpstok_status check_seqs(const fpstok_seqs* s, const char* what);
SeqArgs seq_args(const fpstok_seqs* s);
// A workspace of `need` bytes, 256-byte aligned (NULL if none is needed).
fpstok_status check_ws(size_t need, void* ws, size_t ws_bytes);

}  // namespace fpstok
