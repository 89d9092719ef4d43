// Where the lanes of attend_kernel read, in plain C++: the kernel and a check on
// the host go by the same functions.  es: bytes of an element; ks: a head's size
// in units of 32 elements, as the kernel is built for it; quad = lane / 16,
// l16 = lane % 16; offsets are bytes from the start of a key or a value.
#pragma once

#include <cstdint>

namespace gsi {

// The ks that a head of d elements takes.
constexpr int attend_ks(int d) {
  const int units = (d + 31) / 32;
  return units <= 4 ? units : units <= 6 ? 6 : 8;
}

constexpr int attend_step(int es) { return es == 2 ? 32 : 16; }  // slots
constexpr int key_tiles(int es) { return es == 2 ? 2 : 1; }      // of a step
constexpr int key_pieces(int es, int ks) { return es == 4 ? 2 * ks : ks; }  // of 16 bytes, of a lane

// A lane's piece c is the one at 64 c + 16 quad; from this piece on it may lie
// behind the key, for any size of a head that takes ks.
constexpr int key_guarded(int es, int ks) { return key_pieces(es, ks) - (es == 4 ? 2 : 1) * (ks > 4 ? 2 : 1); }
constexpr bool piece_inside(int es, int d, int c, int quad) { return 64 * c + 16 * quad < d * es; }
// What it reads: behind the key the key's last piece again, which counts as zeros.
constexpr uint32_t piece_at(int es, int ks, int d, int c, int quad) {
  const int at = 64 * c + 16 * quad;
  return c < key_guarded(es, ks) || at < d * es ? at : d * es - 16;
}

// Columns of a value that a lane holds, and the first of them: the last run ends
// with the value.
constexpr int value_columns(int ks) { return 2 * ks; }
constexpr int first_column(int ks, int d, int l16) {
  const int at = l16 * value_columns(ks);
  return at < d - value_columns(ks) ? at : d - value_columns(ks);
}

// A lane's keys (values) of a step lie in one block of 8 slots: the block, and
// the first of its slots; those of a further tile lie 4 slots on.
constexpr int key_block(int es, int l16) { return es == 4 ? l16 >> 3 : l16 >> 2; }
constexpr int key_slot(int es, int l16) { return es == 4 ? l16 & 7 : l16 & 3; }
constexpr int value_slots(int es) { return es == 4 ? 4 : 8; }
constexpr int value_block(int es, int quad) { return es == 4 ? quad >> 1 : quad; }
constexpr int value_slot(int es, int quad) { return es == 4 ? 4 * (quad & 1) : 0; }

// The slot whose page number is read for slot t, of the slots [first, n) in use: no
// other's, and what is read there for a slot outside counts as nothing.
constexpr int slot_in_use(int t, int first, int n) {
  const int at = t > first ? t : first;
  return at < n ? at : n - 1;
}

}  // namespace gsi
