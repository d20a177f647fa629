// The tiled product of two 8-bit tensors: the choice of its tile (fp8_tile.h holds the kernel).
#include "fp8_tile.h"

namespace ifx {
namespace {

typedef Tile<64, 64, 2, 2, 4> TileS;

template <int AF>
hipError_t product(const Fp8Args &a, hipStream_t s)
{
    const int cus = cus_or_default();
    hipError_t e;
    if (a.type != 0 && tiles<TileX>(a, 256) >= cus) return launch_tile<TileX, kFormProduct, AF>(a, s);
    if (launch_middle<kFormProduct, AF>(a, cus, s, &e)) return e;
    // small tiles are bound by what they read from L2 (us, TileG / TileS): 1024 x 2048 x 2048 (256 of TileG) 8.9 / 10.0,
    // to float32 with k 6241 30.8 / 34.2; 300 x 4096 x 4096 (160) 13.8 / 14.8; 512 x 2048 x 2048 (128) 8.6 / 7.4
    if (8 * tiles<TileG>(a, 128) >= 5 * cus) return launch_tile<TileG, kFormProduct, AF>(a, s);
    return launch_tile<TileS, kFormProduct, AF>(a, s);
}

}  // namespace

hipError_t launch_fp8_product(Fp8Args a, hipStream_t s)
{
    a.past = stored_past(a.y, a.m, a.ld_y, a.type == 0 ? 4 : 2);
    return a.a_format ? product<1>(a, s) : product<0>(a, s);
}

}  // namespace ifx
