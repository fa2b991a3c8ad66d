// Decode over an 8-bit cache: e4m3 codes, head_dim 128.
#include "decode_quant.cuh"

namespace lrkv {
template lrkv_status launch_decode_quant_fd<LRKV_Q_E4M3, 128>(const QDecodeParams&, int, int, const void*, const void*,
                                                      const void*, int, int, void*);
}
