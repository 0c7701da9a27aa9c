// How a product of 4-bit matrices is cut into workgroups, chosen by sizes and types.
#pragma once

#include "q4.h"

// How a call is cut into workgroups.
struct q4_shape {
  int tokens;  // a workgroup: 4, 8, 16 or 32 (bf16)
  int rows;    // row blocks a workgroup: 1 or 2 (4 tokens), 1, 2, 4 or 8 (one matrix; fp32 or 32 tokens)
  int splits;  // waves that split the columns
};

/*
 * How a call is cut, from times of graphs of launches (us; rows x columns).
 *   One workgroup for each of the 256 compute units, of as many waves as registers and LDS allow, is best where that cuts
 *   the whole call: so row blocks are shared out one, two or four to a workgroup as their number grows.
 *   One to four tokens.  Up to 256 row blocks one each, sixteen splits (1152 x 13184, one token, 6.5 against 7.0 with eight and
 *   8.7 with four), up to 512 two (5000 x 4096 5.3 against 5.8 with one and four splits, fp32 5.5 against 6.9).  More row
 *   blocks fill the chip with four splits, and from 900 on two a wave keep more bytes in flight for the same waves (16000 x
 *   6016 11.1 against 12.6; 11008 x 4096 7.7 against 7.3).  Under a mask one row block is the unit: 256 of 65536 rows wanted
 *   6.6 against 8.1.
 *   More tokens, 16 at a time; up to eight fetch and cut half of x (3000 x 11008, 6 tokens, 7.4 against 8.5, fp32 13.5 against
 *   17.5).  Up to 256 pairs of row and token blocks one each (1152 x 4096, 16 tokens, 4.8 with sixteen
 *   splits against 5.0 with eight; fp32 8.0 with twelve against 8.7), up to 512 two (4096 x 4096, 32 tokens, 6.2 against 8.0
 *   with one and 8.5 with four; fp32 10.9 against 14.8 and 13.7; gated 9.4 against 10.3 and 11.9).  Then four that share x
 *   (11008 x 4096, 16 tokens, 8.9 against 9.9 with one; gated 12.6 against 13.0), with two splits once that fills the chip (64
 *   tokens 17.4); cutting an fp32 x costs more, so eight share it (8640 x 1856, 29 tokens, 12.6 against 14.5).  Two token tiles
 *   a workgroup (bf16) unpack the codes once for both, in workgroups of twice the work: worth it if enough of these remain,
 *   none is half empty and there are columns to pay for their longer end (28672 x 4096, 64 tokens, 30.6 against 35.4; but
 *   20000 x 4096, 32 tokens, 18.5 against 18.1 and 65536 x 512, 64 tokens, 26.0 against 19.5; gated 11008 x 4096, 32 tokens,
 *   18.2 against 22.3).
 *   A wave gets two column blocks at least: 42752 x 512, one token, 5.4 against 6.0 with one.
 */
inline q4_shape q4_pick_shape(int mt, int kt, int tokens, dbs_dtype xd, bool gated, bool masked) {
  q4_shape p = {};
  if (tokens <= 4) {
    p.tokens = 4;
    p.rows = !gated && !masked && ((mt > 256 && mt <= 512) || mt >= 900) ? 2 : 1;
    p.splits = mt <= 256 * p.rows ? 16 : 4;
  } else {
    const int64_t work = mt * (int64_t)((tokens + 15) / 16);
    const bool whole_pairs = (tokens + 15) / 16 % 2 == 0;
    const bool pairs = xd == DBS_BF16 && whole_pairs && work > (gated ? 1200 : 3000) && kt >= (gated ? 24 : 12);
    p.tokens = pairs ? 32 : tokens <= 8 ? 8 : 16;
    p.rows = work <= 256 ? 1 : work <= 512 ? 2 : !gated && (pairs || (work > 1024 && xd == DBS_F32)) ? 8 : 4;
    if (p.rows == 1) p.splits = xd == DBS_BF16 ? 16 : !gated && kt >= 24 ? 12 : 8;
    else if (p.rows == 2) p.splits = xd == DBS_BF16 && !gated ? 16 : 8;
    else p.splits = p.rows == 4 && work <= 2048 ? 4 : 2;
  }
  while (p.splits > 1 && kt < 2 * p.splits) p.splits /= 2;
  return p;
}
