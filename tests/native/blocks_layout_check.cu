// Host-side check of the block-list decode kernel's shared-memory carve-up for
// every instantiated (D, G, cache type): it fits the 227 KB a block may have at
// every batch size, the regions follow one another without overlap, rings and
// states start on 16 bytes and the pieces' words on 4, and a warp's state fits
// where its ring was.  Built and run by tests/test_blocks_layout.py; no GPU.
#include "decode_blocks.cuh"

#include <cstdio>

using namespace pkv::blk;

template <int D, int G, int KV>
int check()
{
    using C = Cfg<D, G, KV>;
    using S = Smem<D, G, KV>;
    int bad = 0;
    bad += C::STAGE % 16 != 0 || C::TILE_BYTES % 16 != 0 || (C::STATE * 4) % 8 != 0;
    bad += S::STATES != C::W * C::NST * C::STAGE || S::STATES % 16 != 0;
    bad += S::INFO < S::STATES + C::W * C::STATE * 4 || S::INFO % 16 != 0;
    bad += S::TSTART != S::INFO + C::W * C::NST * 16;
    bad += C::NST * C::STAGE < C::STATE * 4;
    bad += C::NT * (C::NT <= 512 ? 1 : 0) != C::NT || 2 * C::W > 32;
    for (int batch : {1, 2, 3, 127, 2047, 2048, 2049, 4095, 4096}) {
        const int words = (S::has_lens(batch) ? 2 : 1) * batch + 1;
        bad += S::meta(batch) < S::TSTART + words * 4 || S::meta(batch) % 16 != 0;
        // pieces [2 W], sums and maxima [2 W], flags [2], edges [6]
        bad += S::total(batch) < S::meta(batch) + (4 * C::W + 8) * 4;
        bad += S::total(batch) > 232448;
    }
    if (bad)
        std::printf("D=%d G=%d KV=%d: %d bad layouts\n", D, G, KV, bad);
    return bad;
}

template <int D, int KV>
int check_groups()
{
    return check<D, 1, KV>() + check<D, 2, KV>() + check<D, 4, KV>() + check<D, 8, KV>();
}

int main()
{
    const int bad = check_groups<64, PKV_F8>() + check_groups<128, PKV_F8>() +
                    check_groups<64, PKV_F16>() + check_groups<128, PKV_F16>() +
                    check_groups<64, PKV_BF16>() + check_groups<128, PKV_BF16>();
    std::printf("blocks layout check: %d bad\n", bad);
    return bad != 0;
}
