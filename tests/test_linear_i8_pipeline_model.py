"""A model of the integer product's barrier hand-offs under random schedules, and its launch plans.

csrc/linear_i8.cu: a producer loads k-blocks into a ring of raw stages, two sets of four converter warps
take the k-blocks in turn and hand two sub-blocks of each to the MMA issuer through four slots.  A
wait tests one parity bit.  A set waits for the k-blocks that it converts alone, so with one full
barrier a stage and an odd number of stages a set comes to a stage whose last k-block was the other
set's and may not have landed: two phases too early, which the bit does not show.  Each stage therefore
has two barriers, by the parity of the lap.

The model replays the roles' loops with the kernel's arithmetic, for one CTA and for a pair; loads
land in any order, commits arrive in order.  Every wait has to pass on the phase that it stands for.
"""
import os
import random
import shutil
import subprocess

import pytest
from test_tc_pipeline_model import Bar, EarlyPass

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_ffn_route_gb300", "csrc")
SLOTS, SET = 4, 4


class Place:
    """I8Place: stage, lap (which barrier), phase of that barrier; n counts k-blocks."""

    def __init__(self, stages, laps):
        self.stages, self.laps, self.s, self.n = stages, laps, 0, 0

    def next(self):
        self.n += 1
        self.s = self.n % self.stages

    @property
    def turn(self):
        return self.n // self.stages

    def barrier(self):  # index, parity, and the phases that have to be complete
        if self.laps == 2:
            return (self.turn & 1, (self.turn >> 1) & 1, (self.turn >> 1) + 1)
        return 0, self.turn & 1, self.turn + 1


def run_schedule(seed, stages, tiles, laps=2, ctas=1, chunk=None):
    """`tiles`: k-blocks of each; `chunk`: sub-blocks an accumulator takes (None: all of a tile's)."""
    rng = random.Random(seed)
    full = [[[Bar(1) for _ in range(stages)] for _ in range(laps)] for _ in range(ctas)]
    empty = [[Bar(SET) for _ in range(stages)] for _ in range(ctas)]
    conv_full = [Bar(SET * ctas) for _ in range(SLOTS)]
    conv_empty = [[Bar(1) for _ in range(SLOTS)] for _ in range(ctas)]
    acc_full = [[Bar(1), Bar(1)] for _ in range(ctas)]
    acc_empty = [Bar(ctas), Bar(ctas)]
    copies, commits = [], []

    def wait(bar, parity, need):
        while not bar.passes(parity):
            yield "blocked"
        if bar.phase < need:
            raise EarlyPass
        assert bar.phase == need, "a wait two phases late never passes for sure"

    def chunks():
        for blocks in tiles:
            n = 2 * blocks
            for k in range(0, n, chunk or n):
                yield min(chunk or n, n - k)

    def producer(c):
        p = Place(stages, laps)
        for blocks in tiles:
            for _ in range(blocks):
                yield from wait(empty[c][p.s], (p.turn & 1) ^ 1, p.turn)
                bar = full[c][p.barrier()[0]][p.s]
                bar.arrive(expect_tx=2)
                copies.extend([bar, bar])  # the weights' and the tokens' part
                p.next()

    def converter(c, mine):
        p, cph, uses = Place(stages, laps), 0, 0
        for blocks in tiles:
            for _ in range(blocks):
                if p.n % 2 == mine:
                    which, parity, need = p.barrier()
                    yield from wait(full[c][which][p.s], parity, need)
                    for h in range(2):
                        slot = 2 * mine + h
                        yield from wait(conv_empty[c][slot], cph ^ 1, uses)
                        yield "step"
                        if h:
                            empty[c][p.s].arrive()
                        conv_full[slot].arrive()
                    cph, uses = cph ^ 1, uses + 1
                p.next()

    def issuer():
        s = 0
        for a, n in enumerate(chunks()):
            yield from wait(acc_empty[a & 1], ((a >> 1) & 1) ^ 1, a >> 1)
            for _ in range(n):
                yield from wait(conv_full[s % SLOTS], (s // SLOTS) & 1, s // SLOTS + 1)
                commits.append([conv_empty[c][s % SLOTS] for c in range(ctas)])
                s += 1
            commits.append([acc_full[c][a & 1] for c in range(ctas)])

    def epilogue(c):
        for a, _ in enumerate(chunks()):
            yield from wait(acc_full[c][a & 1], (a >> 1) & 1, (a >> 1) + 1)
            yield "step"
            acc_empty[a & 1].arrive()

    live = [issuer()] + [r(c) for c in range(ctas) for r in (producer, epilogue)]
    live += [converter(c, m) for c in range(ctas) for m in range(2) for _ in range(SET)]
    blocked = set()
    while True:
        choices = [r for r in live if id(r) not in blocked]
        choices += ["copy"] * (2 if copies else 0) + ["commit"] * (2 if commits else 0)
        if not choices:
            return "deadlock" if live else "ok"
        pick, before, what = rng.choice(choices), Bar.changes, "step"
        if pick == "copy":
            copies.pop(rng.randrange(len(copies))).land()
        elif pick == "commit":
            for bar in commits.pop(0):
                bar.arrive()
        else:
            try:
                what = next(pick)
            except StopIteration:
                live.remove(pick)
        if Bar.changes != before:
            blocked.clear()
        if what == "blocked":
            blocked.add(id(pick))


@pytest.mark.parametrize("stages", range(2, 13))
@pytest.mark.parametrize("ctas", [1, 2])
def test_no_wait_passes_early_with_two_barriers_a_stage(stages, ctas):
    for seed in range(25):
        tiles = [(stages * 3 + seed) % 11 + 1, 2 * stages + 3, 1, stages + seed % 3]
        for chunk in (None, 16):
            assert run_schedule(seed, stages, tiles, ctas=ctas, chunk=chunk) == "ok", (seed, chunk)


def test_with_one_barrier_a_stage_three_stages_pass_early():
    early = {}
    for stages in range(2, 13):
        early[stages] = 0
        for seed in range(60):
            try:
                assert run_schedule(seed, stages, [4 * stages + 5] * 2, laps=1) == "ok"
            except EarlyPass:
                early[stages] += 1
    assert early[3] > 0
    assert all(n == 0 for stages, n in early.items() if stages != 3), early


def run_cpp(tmp_path, body):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text('#include "linear_plan.cuh"\n#include <cstdio>\nusing namespace moe;\n'
                   "int main() {\n" + body + "\n}\n")
    cxx = shutil.which("g++") or shutil.which("c++")
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()


PLAN = """
  const int sms = 152, clusters[3] = {76, 36, 15};
  auto stages_of = [&](const I8Plan &p) {
    return i8_stages(p.mode == kPair ? p.BN / 2 : p.BN, p.mode == kSplit ? i8_exchange(p.BN, p.split) : 0);
  };
"""


def test_every_plan_has_a_ring_that_the_model_covers(tmp_path):
    """Stages of each plan over a sweep of sizes, and the shared memory that they take."""
    out = run_cpp(tmp_path, PLAN + """
  int seen[64] = {};
  for (int few = 0; few < 2; few++)  // clusters as they run, and none known
    for (int R = 9; R < 40000; R += 1 + R / 9)
      for (int N : {16, 512, 1000, 2048, 4096, 7168, 14336})
        for (int K : {16, 512, 2048, 6144, 14336})
          for (int E : {0, 1, 8, 64, 256})
            for (int form = 0; form < 4; form++) {
              const int none[3] = {0, 0, 0};
              const I8Plan p = i8_make_plan(R, N, E, (K + 127) / 128, form & 1, form >> 1, sms,
                                            few ? none : clusters);
              const int s = stages_of(p), x = p.mode == kPair ? p.BN / 2 : p.BN;
              const int ex = p.mode == kSplit ? i8_exchange(p.BN, p.split) : 0;
              if (p.BN < 16 || p.BN > kI8MaxN || p.BN % 16 || p.tiles < 1) return 1;
              if (s < 2 || s > kLinStages) return 1;
              if (s * (kLinM + x) * 128 + kI8Slots * x * 128 + ex > kLinRing) return 1;
              seen[s]++;
            }
  for (int s = 0; s < 64; s++)
    if (seen[s]) printf("%d ", s);""")
    counts = [int(v) for v in out]
    assert min(counts) >= 2 and max(counts) <= 12 and 3 in counts


def test_plans_of_some_sizes(tmp_path):
    """Rows, features, K, experts, gated, fp32 output -> form (0 one CTA a tile, 1 a pair, 2 a split),
    token rows of a tile, split, stages; on 152 SMs."""
    sizes = [(4095, 4096, 14336, 0, 0, 0), (32768, 2048, 6144, 32, 1, 0), (93, 6144, 7168, 0, 0, 0),
             (600, 6144, 2048, 8, 0, 0), (2000, 1000, 8192, 0, 0, 1)]
    calls = "".join(f"""{{ const I8Plan p = i8_make_plan({R}, {N}, {E}, {K} / 128, {g}, {x}, sms, clusters);
  printf("%d/%d/%d/%d ", p.mode, p.BN, p.split, stages_of(p)); }}
""" for R, N, K, E, g, x in sizes)
    assert run_cpp(tmp_path, PLAN + calls) == ["1/192/1/5", "1/192/1/5", "2/96/2/3", "0/160/1/3",
                                               "0/112/1/4"]


def test_the_kernel_waits_on_the_barrier_of_its_lap():
    with open(os.path.join(CSRC, "linear_i8.cu")) as f:
        src = f.read()
    assert "uint64_t raw_full[2][kLinStages];" in src and "&b->full[" not in src
    assert "&b->raw_full[p.lap][p.s]" in src and "ph ^= lap, lap ^= 1" in src
