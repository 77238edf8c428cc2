/*
 * act8.h -- C ABI of libkda_fwd: activations kept in 8 bits between a forward and its backward
 * pass. Conventions as in kda_fwd.h.
 *
 * A row x[0..D) becomes n[i] = round(127 x[i] / m) (ties to even) with m = max |x[i]|, and the
 * scale m / 127; a zero row has scale 0. The value a row holds is n[i] * scale, rounded to the
 * io type (below m = 2^-119 the scale is subnormal and has fewer bits, at last none). A row with a NaN or an infinity gets a NaN scale and comes back as NaN throughout.
 */
#ifndef ACT8_H
#define ACT8_H

#include <stdint.h>

#include "kda_fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* x [rows, D] (io dtype) -> data [rows, D] int8, scale [rows] fp32. D: a multiple of 8, 8 .. 512;
   rows * D below 2^33, at most 2^30 - 64 rows. x and data 16- and 8-byte aligned, scale 4-byte aligned. */
kda_status act8_pack(const void *x, int32_t io, int64_t rows, int32_t D, int8_t *data,
                     float *scale, void *stream);

/* data, scale -> x [rows, D] (io dtype). */
kda_status act8_unpack(const int8_t *data, const float *scale, int32_t io, int64_t rows,
                       int32_t D, void *x, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ACT8_H */
