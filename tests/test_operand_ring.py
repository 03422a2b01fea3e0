"""The ring of unequal operand stages of the products in 16 bits (csrc/operand_ring.h), on the host:
the header's own code is compiled and run through random sequences of tiles, with a consumer that is
any number of stages behind.  Every stage lies inside the ring and on no stage that is still read,
producer and consumer place it alike, barriers' slots and phases are those of the stage, and an empty
ring takes every stage."""
import subprocess

from block_scaled_fp8_persistent_gb300 import build as libbuild

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <random>
#include "operand_ring.h"
using namespace bsfp8::g16;

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

struct Stage { uint32_t at, units, slot, phase; };

int main() {
  std::mt19937 rng(1);
  long long stages = 0, exact_ends = 0, wraps = 0;
  for (int run = 0; run < 3000; ++run) {
    RingPlace producer, consumer;
    RingFill fill;
    std::deque<Stage> live;
    const int most = run % 3 == 0 ? 512 : run % 3 == 1 ? 256 : 64;
    const int lag = (int)(rng() % 11);
    auto consume = [&] {
      uint32_t skipped;
      const Stage s = live.front();
      CHECK(consumer.take(s.units, skipped) == s.at);
      CHECK(consumer.slot == s.slot && consumer.phase == s.phase);
      CHECK(fill.oldest == s.slot && fill.oldest_phase == s.phase);
      consumer.next();
      live.pop_front();
      fill.drop_oldest();
    };
    for (int tile = 0; tile < 40; ++tile) {
      const int height = rng() % 4 == 0 ? most : 1 + (int)(rng() % most);
      const uint32_t units = W_UNITS + half_units(height < 256 ? height : 256) + half_units(height - 256);
      CHECK(units * UNIT >= 4 * 4096u + (height < 256 ? height : 256) / 2 * 128u);
      const int blocks = 1 + (int)(rng() % 12);
      for (int b = 0; b < blocks; ++b, ++stages) {
        uint32_t skipped;
        const bool at_end = producer.head == RING;
        const uint32_t at = producer.take(units, skipped);
        exact_ends += at_end;
        wraps += at == 0;
        while (!fill.fits(units + skipped) || (int)live.size() > lag) {
          CHECK(!live.empty());  // else nothing would ever make room
          consume();
        }
        CHECK(at + units <= RING);
        for (const Stage& s : live) {
          CHECK(at + units <= s.at || s.at + s.units <= at);
          CHECK(s.slot != producer.slot);
        }
        fill.put(units + skipped);
        live.push_back({at, units, producer.slot, producer.phase});
        CHECK(fill.stages == live.size() && fill.stages < MAX_STAGES && fill.used <= RING);
        CHECK(units + skipped < (1u << RingFill::kBits));
        producer.next();
      }
    }
    while (!live.empty()) consume();
    CHECK(fill.used == 0 && fill.sizes == 0);
  }
  CHECK(exact_ends > 100 && wraps > 1000);
  std::printf("%lld stages\n", stages);
}
"""


def test_stages_do_not_meet(tmp_path):
    source, program = tmp_path / "ring.cpp", tmp_path / "ring"
    source.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", "-I" + libbuild.CSRC, str(source), "-o", str(program)], check=True)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
