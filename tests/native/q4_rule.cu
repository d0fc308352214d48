// The rule between folded and scaled weights of the 4-bit tile kernel, and its workspaces.  Host code.
#include "tq_q4_internal.h"

extern "C" int scaled(int m, int group, int mins, long long tiles, int sms) { return tq::q4_scaled_call(m, group, mins != 0, tiles, sms); }
extern "C" int row_tiles(int m, int most) { return (m + tq::q4_tile_rows(m, most) - 1) / tq::q4_tile_rows(m, most); }
extern "C" int scaled_cols(void) { return tq::kQ4ScaledCols; }
extern "C" int tile_cols(void) { return tq::kQ4TileCols; }
