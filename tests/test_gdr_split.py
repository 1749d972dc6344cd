"""Host planning of the divided prefill: csrc/kda_gdr_split.h built alone with g++ (no GPU)."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "linear_attention_serving_prefill_b200", "csrc")

# Reads "num_seqs total_tokens H has_host [offsets]" per case; prints the segment size, then the
# segments of every sequence.
MAIN = r"""
#include <cstdio>
#include <vector>
#include "kda_gdr_split.h"
int main()
{
    int N, T, H, host;
    while (scanf("%d %d %d %d", &N, &T, &H, &host) == 4) {
        std::vector<int32_t> cu(N + 1, 0);
        if (host) for (auto &x : cu) if (scanf("%d", &x) != 1) return 1;
        const kda::SplitBatch b{N, T, H, host ? cu.data() : nullptr};
        const int chunks = kda::plan_split(b);
        printf("%d", chunks);
        if (chunks) for (int n = 0; n < N; ++n) printf(" %d", kda::parts_of(kda::chunks_of(b, n), chunks));
        printf("\n");
    }
}
"""

SMS, MAX_PARTS = 148, 64


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("split")
    (d / "main.cpp").write_text(MAIN)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "main.cpp", "-o", "main"], cwd=d, check=True)

    def run(cases):
        """cases: (lens, H, host offsets given); returns (segment size, segments per sequence) each."""
        lines = []
        for lens, H, host in cases:
            cu = [sum(lens[:i]) for i in range(len(lens) + 1)] if host else []
            lines.append(" ".join(map(str, [len(lens), sum(lens), H, int(host), *cu])))
        out = subprocess.run([str(d / "main")], input="\n".join(lines), text=True, capture_output=True, check=True).stdout
        rows = [list(map(int, r.split())) for r in out.splitlines()]
        assert len(rows) == len(cases)
        return [(r[0], r[1:]) for r in rows]
    return run


def check(lens, H, chunks, parts):
    """What the launches' item lists, CTAs and workspace have room for."""
    if chunks == 0:
        return
    assert max(parts) > 1 and max(parts) <= MAX_PARTS
    assert sum(parts) * H <= SMS, (lens, H, chunks)
    assert sum(2 * p - 3 for p in parts if p > 1) * H <= SMS, (lens, H, chunks)
    assert sum(2 * p - 2 for p in parts) * H <= 2 * SMS, (lens, H, chunks)


def test_one_long_sequence_beside_many_shorter_ones(plans):
    """The segment size that divides the long one evenly would divide all the others too."""
    lens = [90 * 64] + [40 * 64] * 139
    (chunks, parts), = plans([(lens, 1, True)])
    check(lens, 1, chunks, parts)
    lens = [90 * 64, 40 * 64]
    (chunks, parts), = plans([(lens, 32, True)])
    check(lens, 32, chunks, parts)


@pytest.mark.parametrize("seed", range(4))
def test_every_split_fits_the_device(plans, seed):
    rng = random.Random(seed)
    cases = []
    for _ in range(2000):
        H = rng.choice([1, 1, 1, 2, 3, 4, 8, 16, 32, 49, 74])
        N = rng.randint(1, max(1, SMS // H - 1))
        kind = rng.randrange(3)
        if kind == 0:
            lens = [rng.randint(0, 9000) for _ in range(N)]
        elif kind == 1:
            lens = [rng.choice([1000, 2500, 2560, 40])] * N
        else:
            lens = [int(2 ** rng.uniform(0, 16)) for _ in range(N)]
        lens[rng.randrange(N)] = rng.randint(1, 60000)
        cases.append((lens, H, rng.random() < 0.8))
    got = plans(cases)
    for (lens, H, _), (chunks, parts) in zip(cases, got):
        check(lens, H, chunks, parts)
    assert any(c for c, _ in got) and not all(c for c, _ in got)
