"""How attention cuts a call, worked out on the host from the sizes that a caller
gives, without a GPU: a small program around the plan's own header says which
sequences go by tiles of 16 rows, which by more, and what their sums take of the
workspace."""

import random
import subprocess

import pytest

import tenant_linear_layers_amd as T
from tenant_linear_layers_amd import build

PROGRAM = r"""
#include <cstdio>
#include "attention_plan.h"
namespace bd { Divisor divisor(int by) { return Divisor{1, 0, by}; } }
int main() {
  bd::AttnArgs a{};
  int bits;
  while (scanf("%d %d %d %d %d %d %d %d %d", &a.tokens, &a.seqs, &a.max_q, &a.heads, &a.kv_heads,
               &a.dim, &a.width, &a.page, &bits) == 9) {
    a.group = a.heads / a.kv_heads;
    a.bits = bits;
    const bd::Way w = bd::way_of(a);
    printf("%d %d %d %d %d %d %zu %zu\n", w.cut[0].R, w.cut[1].R, w.cut[0].most, w.cut[1].least,
           w.items[0], w.items[1], w.bytes[0], w.bytes[1]);
  }
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.hip").write_text(PROGRAM)
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-O3", "-Wall")]
    subprocess.run([build.hipcc(), *flags, "-O1", "-w", str(at / "plan.hip"), "-o",
                    str(at / "plan")], check=True, capture_output=True)

    def run(calls):
        """(tokens, seqs, max_q, heads, kv_heads, dim, width, page, bits) of each."""
        out = subprocess.run([str(at / "plan")], input="\n".join(" ".join(map(str, c))
                                                                 for c in calls),
                             text=True, capture_output=True, check=True).stdout
        names = "few many most least few_items many_items few_bytes many_bytes".split()
        return [dict(zip(names, map(int, line.split()))) for line in out.splitlines()]
    return run


def _call(new, kv, heads, kv_heads, dim, page, bits=4):
    width = max(-(-m // page) for m in kv)
    return (sum(new), len(new), max(new), heads, kv_heads, dim, width, page, bits)


ALL = 2 ** 31 - 1
WAYS = [
    # new, kv, heads, kv_heads, dim, most rows of a sequence by 16, rows of the others' tiles
    ([1] * 40, [8000] * 40, 64, 8, 128, 32, 0),
    ([4] * 16, [4000] * 16, 64, 8, 128, 32, 0),
    ([4] * 16 + [200], [4000] * 17, 64, 8, 128, 32, 128),
    ([4] * 16 + [200], [4000] * 17, 64, 8, 64, 32, 128),
    ([4] * 40 + [100], [8000] * 41, 64, 8, 128, 32, 64),
    ([2] * 20 + [4] * 20 + [100], [4000] * 41, 64, 8, 128, 32, 64),
    ([3, 100, 4, 1], [900, 2000, 700, 5000], 64, 8, 64, 32, 128),
    ([4] * 100 + [100], [1000] * 101, 64, 8, 128, 16, 64),   # by 32 it would not fit
    ([1, 40], [150, 90], 8, 8, 128, ALL, 0),                 # 32 tiles in all
    ([20, 20], [200, 200], 8, 2, 128, ALL, 0),
    ([16], [8000], 64, 8, 128, ALL, 0),
    ([40], [90], 64, 64, 128, 0, 64),
    ([2048], [2048], 64, 8, 128, 0, 128),
    ([70, 40], [70, 300], 64, 64, 128, 32, 64),
    ([200], [500], 64, 16, 64, 0, 128),
    ([40, 70], [90, 150], 64, 64, 128, 32, 64),
    ([200], [500], 64, 16, 128, 0, 128),
]


@pytest.mark.parametrize("new,kv,heads,kv_heads,dim,by16,rows", WAYS)
def test_which_rows_go_by_16(plan, new, kv, heads, kv_heads, dim, by16, rows):
    w, = plan([_call(new, kv, heads, kv_heads, dim, 64)])
    assert w["few"] == (16 if by16 else 0) and w["many"] == rows
    if by16:
        assert w["most"] == by16
    if by16 and rows:
        assert w["least"] == by16


def test_no_plan_needs_more_than_the_size_asked_for(plan):
    """Whatever the cache's type is, which the size query does not know."""
    rng = random.Random(4)
    calls = []
    for _ in range(4000):
        group = rng.choice([1, 2, 4, 7, 8, 14, 16, 32, 64])
        kv_heads = rng.choice([1, 2, 4, 8, 16, 64][:6 if group <= 16 else 3])
        seqs = int(2 ** rng.uniform(0, 12))
        max_q = int(2 ** rng.uniform(0, 13))
        tokens = min(int(seqs * max_q * rng.uniform(0.01, 1)) + max_q, seqs * max_q, 2 ** 18)
        dim, page = rng.choice([64, 128]), rng.choice([16, 64, 128])
        width = int(2 ** rng.uniform(0, 17)) // page + 1
        calls += [(tokens, seqs, max_q, group * kv_heads, kv_heads, dim, width, page, bits)
                  for bits in (4, 8, 16)]
    for c, w in zip(calls, plan(calls), strict=True):
        need = T.paged_attention_workspace_size(*c[:8])
        assert w["few_bytes"] + w["many_bytes"] <= need, c
        for part, rows in (("few", w["few"]), ("many", w["many"])):
            bytes_of = w[part + "_items"] * rows * (c[5] + 2) * 4
            assert w[part + "_bytes"] in (0, bytes_of), c
