"""The counted waits of the tiled product's ring of LDS stages, checked in a
host program against csrc/copy_ring.h: a stage may only be read once all of
its copies have landed.  Needs no GPU."""
import os
import re
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "int4_routed_expert_router_amd", "csrc")


def _value(expr, copies, scaled):
    expr = expr.replace("SCALED", "scaled")
    expr = re.sub(r"\((\w+) \? (\d+) : (\d+)\)", r"(\2 if \1 else \3)", expr)
    return eval(expr, {"__builtins__": {}}, {"LD": copies, "scaled": scaled})


def test_waits_of_the_ring(tmp_path):
    # the counts that the kernel waits for, and whether its prologue uses the first
    text = open(os.path.join(CSRC, "project.hip")).read()
    first, each = re.search(r"constexpr int kFirst = ([^,;]+), VM = ([^;]+);", text).groups()
    assert "s_waitcnt(0x0F70 | kFirst)" in text and "s_waitcnt(0x0070 | (VM & 15))" in text
    copies = 6  # 384 rows of 128 bytes over eight wavefronts, eight rows to a copy
    (tmp_path / "ring.cpp").write_text('''
#include <cstdio>
#include <cstdlib>
#include "copy_ring.h"
int main(int n, char **v) {
  for (int i = 1; i + 3 < n; i += 4)
    std::printf("%d", coli::ring_waits_hold(std::atoi(v[i]), std::atoi(v[i + 1]), std::atoi(v[i + 2]),
                                            std::atoi(v[i + 3])));
}
''')
    exe = str(tmp_path / "ring")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(tmp_path / "ring.cpp"), "-o", exe],
                   check=True)

    def hold(*rows):
        args = [str(int(v)) for r in rows for v in r]
        out = subprocess.run([exe, *args], check=True, capture_output=True, text=True).stdout
        return [c == "1" for c in out]

    assert hold(*[(copies, s, _value(first, copies, s), _value(each, copies, s))
                  for s in (False, True)]) == [True, True]
    # what the counts guard against: the first step's wait is one short after
    # two stages in flight, and one more in any step is too many
    assert hold((copies, True, 2 * copies, copies + 1), (copies, True, copies, copies + 2),
                (copies, False, 2 * copies, copies + 1)) == [False, False, False]
    assert hold((copies, False, 2 * copies, copies), (copies, True, 2 * copies, copies)) == [True, True]
