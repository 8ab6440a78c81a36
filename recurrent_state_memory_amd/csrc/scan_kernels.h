// scan_kernels.h -- launch interface of the channelwise recurrence.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_scan.h"

namespace gdr {
namespace scan {

constexpr int kTileC = 64;      // channels of a tile
// Waves of a full tile, one block of tokens each.  A tile costs about a microsecond
// besides its elements (the ticket, the joins), and only workgroups of their own
// overlap one tile's loads with another's arithmetic: forward with 4 / 8 / 16 waves
// 134 / 119 / 128 us on 8 x 4096 x 2048 bf16 gated and 129 / 103 / 109 on 1 x 32785 x
// 2048 with given decays; backward with 2 / 4 / 8 waves 257 / 241 / 287 gated (the same
// with fewer registers: 4 / 8 waves 227 / 236).
constexpr int kFwdWaves = 8;
constexpr int kBwdWaves = 4;
constexpr int kSuper = 8;       // tiles that share one hand-over along the sequence (16: no faster)

// Chains that are worked on together.  32 chains of 16 tiles under way read whole
// rows of few batch rows, which HBM serves faster than rows of many at once; where
// the gates' arithmetic bounds the kernel and not HBM, the more chains, the fewer
// waits for a tile before.  8 x 4096 x 2048, teams of 32 against 128: decays given,
// forward 107 / 113 us, backward 181 / 192; fp32 gated backward (half the batch) 186
// / 194; bf16 gated backward 248 / 242, forward 120 / 118 us.
constexpr int team_of(bool alpha, int io_dtype) { return alpha || io_dtype != GDR_BF16 ? 32 : 128; }

constexpr size_t blocks_of(int T) { return ((size_t)T + GDR_SCAN_BLOCK - 1) / GDR_SCAN_BLOCK; }
constexpr size_t tiles_t(int T, int waves) { return (blocks_of(T) + waves - 1) / waves; }
constexpr size_t chains_of(int B, int C) { return (size_t)B * ((C + kTileC - 1) / kTileC); }
// A launch has fewer than 2^23 tiles (a grid holds 2^32 threads).
constexpr size_t kMaxTiles = (size_t)1 << 23;
constexpr bool too_many_tiles(int B, int T, int C) { return chains_of(B, C) * tiles_t(T, kBwdWaves) >= kMaxTiles; }

// Which tile the number drawn stands for: chains are taken in teams, and within a team
// the first tiles of all its chains come before the second ones, so a tile's number is
// larger than those of the tiles before it in its chain.  There are nchain * nt numbers;
// one behind them, which only a ticket that another call draws from as well can give,
// stands for no tile (chain -1).
struct Turn {
  int chain, tt;   // chain, and the tile's place along it in the order of joining
};
__host__ __device__ constexpr Turn turn_of(uint32_t number, int nchain, int nt, int team_size) {
  if (number >= (uint32_t)nchain * (uint32_t)nt) return Turn{-1, 0};
  const uint32_t full = (uint32_t)team_size * (uint32_t)nt, team = number / full, in = number - team * full;
  const uint32_t left = (uint32_t)nchain - team * (uint32_t)team_size;   // of the last team
  const uint32_t size = left < (uint32_t)team_size ? left : (uint32_t)team_size, tt = in / size;
  return Turn{(int)(team * (uint32_t)team_size + (in - tt * size)), (int)tt};
}

// Workspace of the forward and of the backward (bytes; 0: none needed).
size_t fwd_workspace(int B, int T, int C);
size_t bwd_workspace(int B, int T, int C, bool gated, bool ckpt);

// Arguments already checked; a.workspace large enough.
hipError_t launch_scan_fwd(const gdr_scan_args& a, hipStream_t s);
hipError_t launch_scan_bwd(const gdr_scan_bwd_args& a, hipStream_t s);
hipError_t launch_scan_step(const gdr_scan_step_args& a, hipStream_t s);

// The hand-over words of the chains, and the ticket, at the start of a workspace.
struct Chains {
  uint32_t* ticket;    // NULL: one tile per chain, nothing is handed over
  uint64_t* tiles;     // [chains][tiles][64] each tile's map of the state
  uint64_t* supers;    // [chains][supers][64] the state before each super
};
size_t chain_bytes(int B, int T, int C, int waves);   // a multiple of 256
Chains chains_at(void* workspace, int B, int T, int C, int waves);
// No word written, and the tickets at 0, before the kernels that use them.
hipError_t clear_chains(void* workspace, size_t bytes, hipStream_t s);

// The forward of the backward's inputs that writes the block-start states alone (its
// chains cleared).
hipError_t launch_ckpt(const gdr_scan_bwd_args& a, float* ckpt, void* workspace, hipStream_t s);

// Whether rows and buffers allow four channels at a time.
inline bool vec4_ok(const void* p, size_t elem) { return (reinterpret_cast<uintptr_t>(p) & (4 * elem - 1)) == 0; }

}  // namespace scan
}  // namespace gdr
