// Internal interface of the layer operators' translation units.
#pragma once

#include "internal.h"

namespace mbt {

// (mbtile_host.cpp)  2-D tiled map over `rows` rows of `row_bytes` bytes, `ld`
// bytes apart: box = 128 bytes x box_rows rows, 128-byte swizzle, zero fill.
int encode_bytes_map(CUtensorMap *map, const void *src, int64_t rows, int64_t row_bytes, int64_t ld,
                     int box_rows);
// (mbtile_host.cpp)  Address of the current device's status word, looked up once per device.
int device_status_word(int32_t **word);

}  // namespace mbt
