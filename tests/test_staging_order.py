"""The order of bulk copies and writes in the cross entropy's staging buffers
(csrc/staging.h, compiled alone): no buffer is written while a copy that reads
it may be under way, whichever kinds of tiles follow one another."""
import subprocess

from _host_cxx import compile_host

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <deque>
#include "staging.h"

// Copy groups that may not have read their buffers yet (a bit per buffer), the
// slowest that the waits allow.
std::deque<int> unread;
int open_group = 0;

struct Slow {
  template <int N> void wait_read() {
    while ((int)unread.size() > N) unread.pop_front();
  }
  void commit() {
    unread.push_back(open_group);
    open_group = 0;
  }
};

moe::StagingTurns<Slow> turns;
int faults = 0;

void write(int buffers) {
  for (int g : unread) faults += (g & buffers) != 0;
}
void box(int buffer, bool stored) {          // as store_boxes
  if (stored) {
    turns.before_box();
    write(buffer);
    open_group = buffer;
  }
  turns.after_box();
}
void both() {                                // as dX's fp32 sums
  turns.before_both();
  write(3);
  open_group = 3;
  turns.after_both();
}

int main() {
  int after_both = 0;
  for (int seed = 0; seed < 2000; ++seed) {
    std::srand(seed);
    unread.clear();
    bool was_both = false;
    for (int tile = 0; tile < 12; ++tile) {
      const int kind = std::rand() % 3, turns_of_tile = 1 + std::rand() % 4;
      for (int i = 0; i < turns_of_tile; ++i) {
        if (kind == 0) {
          both();
          was_both = true;
        } else {
          after_both += was_both;
          was_both = false;
          box(1, std::rand() % 4 != 0);
          box(2, std::rand() % 4 != 0);
        }
      }
    }
  }
  std::printf("%d %d\n", faults, after_both);
}
"""


def test_no_buffer_is_written_while_it_is_read(tmp_path):
    out = subprocess.run([compile_host(tmp_path, PROGRAM)], capture_output=True, text=True, check=True).stdout
    faults, after_both = map(int, out.split())
    assert after_both > 1000                  # dW tiles behind dX tiles
    assert faults == 0
