// Arguments of the linear attention kernels, shared by their launchers.
#pragma once

#include <stdint.h>

namespace mssm {
namespace la {

// One of the tensors as a pass reads it: token rows `row` elements apart, the
// values of head h / div at (h / div) * its head size.
struct View {
  const void* p = nullptr;
  int64_t row = 0;
  int div = 1;
};

// Where sequences and their segments lie.
struct Grid {
  const int64_t* offsets = nullptr;  // [seqs + 1], or null: dense [seqs, L]
  int64_t seqs = 0, L = 0;           // L: tokens of a dense sequence
  int64_t tokens = 0;                // in all
  int64_t segs = 1;                  // segments of a dense sequence
  int64_t seg_len = 0;               // tokens of a segment
  int64_t slots = 0;                 // segment slots in all
};

struct PassArgs {
  Grid grid;
  View x, y, z, e;
  const float* g = nullptr;          // log decays
  int64_t g_row = 0;                 // heads, or 0: one for each head
  int heads = 0;
  bool paired = false;               // two heads a block: they share x and y, dB <= 64
  int dA = 0, dB = 0;                // sizes of x, y and of z, out
  float scale = 1.0f;
  // states, element (a, b) at a * sA + b * sB of a head's dA * dB
  int64_t sA = 0, sB = 0;
  const float* init = nullptr;       // [seqs, heads, ..], or null: zero
  float* last = nullptr;             // [seqs, heads, ..], or null
  const float* seg_states = nullptr; // [slots, heads, ..]: the state each segment starts from
  // state-only passes
  float* seg_out = nullptr;          // [slots, heads, ..]: each segment's own state
  float* seg_decay = nullptr;        // [slots, heads]
  // output
  void* out = nullptr;               // [tokens, heads, dB], of the inputs' type
  bool out_f32 = false;              // dq, dk: float32 instead
  // gradient of the log decays: written by dq, read by dk
  float* u = nullptr;                // [tokens, heads]
  float* q_sums = nullptr;           // [a segment's chunks, heads, 4]: a wavefront's part each
  float* dumps = nullptr;            // [a segment's dumps, heads, ..]: states as dq holds them
  // A segment's chunks and dumps (one for every 256 tokens begun) lie from slot times
  // these on, with by_token also its first token / C (/ 256) further.
  int64_t chunks_per_slot = 0, dumps_per_slot = 0;
  bool by_token = false;
  // written by dk
  float* dg = nullptr;               // [tokens, heads], or null
  float* head_part = nullptr;        // [slots, heads]: sums of dg, or null
};

}  // namespace la
}  // namespace mssm
