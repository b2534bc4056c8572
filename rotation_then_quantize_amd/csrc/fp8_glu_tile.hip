// fp8_glu_tile.hip -- the gated feed-forward's product for outputs of few tiles: 32, 64 or 128 tokens by 128 channels per
// workgroup.
//
// 8 waves in 2 x 4, each BM / 2 tokens by 32 channels and their partners, laid as in the large kernel.  A ring of three LDS
// stages of one block of the reduction each, loaded three stages ahead; a block's fragments are read while the block before
// it is multiplied.  The tokens' and the two weights' scales, of kTable blocks at a time, are put into LDS beforehand.  The
// outputs' staging takes the ring's place.
//
// Bound by LDS where the weights are in the caches: a stage of 64 tokens writes 40 KB and reads 96, in 0.55-0.6 us, one of 32
// writes 36 and reads 80, in 0.5 (1.1 and more where they come from HBM and fill the CUs: 64 x 4096, 16384 channels).  Four
// waves with larger tiles, which read 64 KB for 64 tokens, have twice the loads each to issue and took 0.95 us.  Weights straight
// into registers, where no other wave needs them (8 waves of 16 channels each), took 1 us: the instruction's operand is 16 rows,
// so that a load touches half of 16 lines of 128 bytes, and each line is touched twice.  bf16 products of the decoded codes
// (fp8_glu_small.hip) take 1.3 to 1.7 times the time here.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_glu.h"
#include "fp8_internal.h"
#include "rtq_internal.h"

namespace rtq {
namespace {

using namespace fp8;

constexpr int kChannels = 128, BN = 2 * kChannels, kSlots = 3;
constexpr int kWavesM = 2, kWavesN = 4, kWaves = kWavesM * kWavesN, kThreads = 64 * kWaves;
constexpr int kTable = 16;   // blocks whose scales are in LDS (an even number)

template <int BM>
constexpr int tile_lds() { return kSlots * (BM + BN) * BK + kTable * (BM + 2) * static_cast<int>(sizeof(float)) + kGluScales; }

template <int BM, bool kE8M0>
__global__ void __launch_bounds__(kThreads)
glu_tile_kernel(GluParams p) {
    constexpr int WM = BM / kWavesM, TM = WM / 16, TN = 4;
    constexpr int kABytes = BM * BK, kStage = kABytes + BN * BK;
    constexpr int kALoads = BM < 64 ? 1 : BM / 8 / kWaves, kWLoads = BN / 8 / kWaves, kLoads = kALoads + kWLoads;   // 1 KB loads per wave
    constexpr int kARows = BM < 64 ? BM / kWaves : 8;   // of a load: 32 tokens are half a load each
    static_assert(kGluStage <= kSlots * kStage, "the outputs' LDS");
    extern __shared__ __attribute__((aligned(1024))) uint8_t lds[];
    const uint32_t lds_base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(lds));
    float* table = reinterpret_cast<float*>(lds + kSlots * kStage);   // [block][token], then [block][gate, partner]
    float* w_table = table + kTable * BM;
    GluLds out_lds{lds, reinterpret_cast<uint32_t*>(w_table + 2 * kTable)};

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWavesN, wn = wave % kWavesN;
    const int g = lane >> 4, l15 = lane & 15;

    // 8 contiguous ranges of tiles, one per XCD (workgroup b runs on XCD b % 8), a column's tiles next to each other
    const int total = p.tiles_t * p.tiles_n, per = (total + 7) / 8;
    const int b = static_cast<int>(block_index()), local = b / 8, lin = b % 8 * per + local;
    if (local >= per || lin >= total) return;
    const int64_t m0 = static_cast<int64_t>(lin % p.tiles_t) * BM;
    const int n0 = lin / p.tiles_t * kChannels;
    const int blocks = (p.K + BK - 1) / BK;

    const int rows_a = static_cast<int>(min<int64_t>(BM, p.T - m0));
    const int second = wave >= kWaves / 2 ? 1 : 0;   // this wave loads the other projection's rows
    const v4i rsa = make_rsrc(p.x + m0 * p.K, static_cast<uint32_t>(rows_a) * static_cast<uint32_t>(p.K));
    const v4i rsw = make_rsrc(p.w + (static_cast<int64_t>(second) * p.N + n0) * p.K, static_cast<uint32_t>(kChannels) * static_cast<uint32_t>(p.K));

    // LDS rows of 128 bytes, chunk c (16 bytes) of row r at chunk c ^ ((r >> 1) & 7); LDS weight row 64 q + 16 j + l is
    // channel 32 q + 16 (j % 2) + l of the gate (j < 2) or of its partner.
    const int kcol = ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7)) << 4;
    const int a_row = kARows * wave + (lane >> 3), a_kcol = ((lane & 7) ^ ((a_row >> 1) & 7)) << 4;
    const uint32_t a_off = static_cast<uint32_t>(a_row * p.K + a_kcol);
    const uint32_t w_off = static_cast<uint32_t>((8 * (wave % (kWaves / 2)) + (lane >> 3)) * p.K + kcol);
    const uint32_t a_step = static_cast<uint32_t>(8 * kWaves * p.K), w_step = a_step / 2;
    auto issue = [&](int kb, int slot) {
        const uint32_t base = lds_base + static_cast<uint32_t>(slot * kStage + wave * 1024);
        auto from = [&](int col) { return kb * BK + col < p.K ? static_cast<uint32_t>(kb * BK) : kOob; };   // zeros past the row's end
        const uint32_t k0 = from(kcol);
        if constexpr (kARows < 8) {
            if (lane < 8 * kARows) load_to_lds(rsa, a_off + from(a_kcol), base - wave * 1024 + wave * kARows * BK);
        } else {
#pragma unroll
            for (int q = 0; q < kALoads; ++q) load_to_lds(rsa, a_off + q * a_step + k0, base + q * kWaves * 1024);
        }
#pragma unroll
        for (int q = 0; q < kWLoads; ++q) load_to_lds(rsw, w_off + q * w_step + k0, base + kABytes + q * kWaves * 1024);
    };
    auto fill = [&](int c0) {   // the tables of blocks c0 ..; token r of wave-row wm at [block][wm][r % 16][r / 16]
#pragma unroll 2
        for (int e = tid; e < kTable * BM; e += kThreads) {
            const int kb = min(c0 + e / BM, blocks - 1), r = e % BM;
            const int64_t m = min<int64_t>(m0 + r, p.T - 1);
            table[e / BM * BM + (r / WM * 16 + (r & 15)) * TM + (r % WM >> 4)] = load_scale<kE8M0>(p.x_scale, kb * p.T + m);
        }
        if (tid < 2 * kTable) {
            const int kb = min(c0 + tid / 2, blocks - 1);
            w_table[tid] = load_scale<kE8M0>(p.w_scale, static_cast<int64_t>((tid % 2 * p.N + n0) / kFp8Block) * blocks + kb);
        }
    };
    const uint32_t f0 = static_cast<uint32_t>(l15 * BK + ((g ^ (l15 >> 1)) << 4));
    const uint32_t f1 = static_cast<uint32_t>(l15 * BK + (((g + 4) ^ (l15 >> 1)) << 4));
    auto read_frag = [&](const uint8_t* base) {
        const v4i x = *reinterpret_cast<const v4i*>(base + f0), y = *reinterpret_cast<const v4i*>(base + f1);
        return v8i{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    };

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
    v8i fa[2][TM], fw[2][TN];
    float sc[2][TM], sw[2][2];
    auto read_scales = [&](auto set, int kb) {
        constexpr int P = decltype(set)::value;
#pragma unroll
        for (int i = 0; i < TM; ++i) sc[P][i] = table[kb % kTable * BM + (wm * 16 + l15) * TM + i];
        sw[P][0] = w_table[kb % kTable * 2];
        sw[P][1] = w_table[kb % kTable * 2 + 1];
    };
    auto read = [&](auto set, int kb, int slot) {
        constexpr int P = decltype(set)::value;
#pragma unroll
        for (int j = 0; j < TN; ++j) fw[P][j] = read_frag(lds + slot * kStage + kABytes + (wn * 64 + j * 16) * BK);
#pragma unroll
        for (int i = 0; i < TM; ++i) fa[P][i] = read_frag(lds + slot * kStage + (wm * WM + i * 16) * BK);
        read_scales(set, kb);
    };
    // Block kb (in slot `slot`) from the fragments and scales of set P, while those of block kb + 1 are read into the other.
    // Nothing here is conditional: with a branch the compiler would wait for all of the reads before the products.  Past the
    // last block zeros are loaded, and what is read is not used.
    auto block = [&](auto set, int kb, int slot, int next) {
        constexpr int P = decltype(set)::value;
        lds_done();                            // this wave's fragments of block kb are in registers
        wait_vmcnt<(kSlots - 2) * kLoads>();   // block kb + 1 has landed (later ones may be in flight) ...
        barrier();                             // ... in every wave; block kb's slot is free
        issue(kb + kSlots, slot);
        read(std::integral_constant<int, 1 - P>{}, kb + 1, next);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const float s[2] = {sc[P][i] * sw[P][0], sc[P][i] * sw[P][1]};
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const v4f d = mfma<false>(fw[P][j], fa[P][i], v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s[j / 2], acc[i][j][r]);
            }
        }
    };
    constexpr auto P0 = std::integral_constant<int, 0>{};
    constexpr auto P1 = std::integral_constant<int, 1>{};
#pragma unroll
    for (int s = 0; s < kSlots; ++s) issue(s, s);
    fill(0);
    if (tid < 2 * kGluSet) out_lds.scales[tid] = 0u;
    wait_vmcnt<(kSlots - 1) * kLoads>();
    lds_done();
    barrier();
    read(P0, 0, 0);
    int slot = 0;
    auto after = [&](int s) { return s + 1 < kSlots ? s + 1 : 0; };
    for (int c0 = 0; c0 < blocks; c0 += kTable) {
        if (c0 != 0) {   // the next blocks' scales, once every wave has read the last of the old ones
            lds_done();
            barrier();
            fill(c0);
            lds_done();
            barrier();
            read_scales(P0, c0);
        }
        const int c1 = min(c0 + kTable, blocks);
        int kb = c0;
        for (; kb + 1 < c1; kb += 2) {
            const int s1 = after(slot), s2 = after(s1);
            block(P0, kb, slot, s1);
            block(P1, kb + 1, s1, s2);
            slot = s2;
        }
        if (kb < c1) block(P0, kb, slot, after(slot));
    }
    wait_vmcnt<0>();   // nothing is still writing the LDS that the outputs go through ...
    lds_done();
    barrier();         // ... nor reading it, in any wave
    glu_tile_outputs<WM, kE8M0>(p, acc, m0, n0, wm, wn, tid, out_lds);
}

template <int BM>
hipError_t launch(GluParams p, bool e8m0, hipStream_t stream) {
    auto kernel = e8m0 ? glu_tile_kernel<BM, true> : glu_tile_kernel<BM, false>;
    int per_cu = 0;
    const hipError_t e = kernel_blocks_per_cu(reinterpret_cast<const void*>(kernel), kThreads, tile_lds<BM>(), &per_cu);
    if (e != hipSuccess) return e;
    p.tiles_t = static_cast<int>((p.T + BM - 1) / BM);
    p.tiles_n = p.N / kChannels;
    const int64_t total = static_cast<int64_t>(p.tiles_t) * p.tiles_n;
    kernel<<<grid_of((total + 7) / 8 * 8), kThreads, tile_lds<BM>(), stream>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_glu_tile(const GluParams& p, bool e8m0, int tokens, hipStream_t stream) {
    return tokens == 32 ? launch<32>(p, e8m0, stream) : tokens == 64 ? launch<64>(p, e8m0, stream) : launch<128>(p, e8m0, stream);
}

}  // namespace rtq
