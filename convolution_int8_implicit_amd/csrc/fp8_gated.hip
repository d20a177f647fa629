// The tiled gated pair of projections, its 8-bit form and its gradient: the choice of their tiles (fp8_tile.h holds the
// kernel).
#include "fp8_tile.h"

namespace ifx {
namespace {

// To codes: a block of 128 columns of the result a tile.
typedef Tile<64, 256, 2, 2, 3> TileC;
typedef Tile<128, 256, 4, 2, 3> TileD;

template <int FORM>
hipError_t gated(const Fp8Args &a, hipStream_t s)
{
    const int cus = cus_or_default();
    if constexpr (FORM == kFormGated8) {
        if (tiles<TileX>(a, 128) >= cus) return launch_tile<TileX, FORM, 0>(a, s);
        // while all of the smaller tiles run at once (us, TileD / TileC): 100 x 8192 x 2048 (128 of TileC) 15.2 / 13.4,
        // 2000 x 1000 x 500 (256) 8.5 / 8.3, 300 x 8192 x 2048 (320) 16.2 / 28.0, 1000 x 4096 x 4096 (512) 32.5 / 46.1
        return tiles<TileC>(a, 128) <= cus ? launch_tile<TileC, FORM, 0>(a, s) : launch_tile<TileD, FORM, 0>(a, s);
    } else {
        hipError_t e;
        if (a.type != 0 && tiles<TileX>(a, 128) >= cus) return launch_tile<TileX, FORM, 0>(a, s);
        if (launch_middle<FORM, 0>(a, cus, s, &e)) return e;
        return launch_tile<TileG, FORM, 0>(a, s);
    }
}

}  // namespace

hipError_t launch_fp8_gated(Fp8Args a, Fp8Mode mode, hipStream_t s)
{
    const int bytes = a.type == 0 ? 4 : 2;
    a.past = !a.codes && stored_past(a.y, a.m, a.ld_y, bytes) && (mode != kGatedGrad || stored_past(a.y2, a.m, a.ld_y2, bytes));
    if (mode == kGatedGrad) return gated<kFormGrad>(a, s);
    return a.codes ? gated<kFormGated8>(a, s) : gated<kFormGated>(a, s);
}

}  // namespace ifx
