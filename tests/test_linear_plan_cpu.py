"""How the epilogue's gradient is dealt out (csrc/linear_plan.h), compiled for the host: clusters of more CTAs than every device promises
to place only where the device holds all of them at once."""
import json
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "persistent_tile_scheduled_gb300", "csrc")
ROWS, EXPERTS, COLUMNS = (0, 1, 127, 1000, 1023, 1024, 2048, 9115, 16384, 1 << 20), (1, 2, 8, 64), (8, 32, 256, 264, 512, 600, 616, 1024, 2048, 7000, 8192, 32776)
SMS, ROOMS = (8, 132, 152), (-1, 0, 1, 16)

PROGRAM = r"""
#include <cstdio>
#include "linear_plan.h"
int main() {
    const long long rows[] = {%ROWS%}, experts[] = {%EXPERTS%}, columns[] = {%COLUMNS%}, sms[] = {%SMS%}, rooms[] = {%ROOMS%};
    bool first = true;
    printf("[");
    for (long long r : rows) for (long long e : experts) for (long long n : columns) for (long long s : sms) for (long long room : rooms)
        for (int gated = 0; gated < 2; ++gated) for (int dbias = 0; dbias < 2; ++dbias) {
            const pts::GradShape g = pts::grad_shape(r, e, n, gated, dbias, static_cast<int>(s), static_cast<int>(room));
            printf("%s[%lld, %lld, %lld, %lld, %lld, %d, %d, %d, %d, %d, %lld, %lld]", first ? "" : ",\n", r, e, n, s, room, gated, dbias, g.tx, g.threads, g.ctas,
                   (long long)g.blocks, (long long)g.units);
            first = false;
        }
    printf("]\n");
    return 0;
}
"""


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is needed to compile the host program")
    d = tmp_path_factory.mktemp("plan")
    src = PROGRAM
    for name, values in (("ROWS", ROWS), ("EXPERTS", EXPERTS), ("COLUMNS", COLUMNS), ("SMS", SMS), ("ROOMS", ROOMS)):
        src = src.replace(f"%{name}%", ", ".join(map(str, values)))
    (d / "plan.cpp").write_text(src)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True, capture_output=True)
    out = json.loads(subprocess.run([str(d / "plan")], check=True, capture_output=True, text=True).stdout)
    return {tuple(x[:7]): tuple(x[7:]) for x in out}


def test_no_cluster_is_larger_than_the_device_places(shapes):
    larger = 0
    for (rows, experts, N, sms, room, gated, dbias), (tx, threads, ctas, blocks, units) in shapes.items():
        if dbias:   # (else no cluster is formed)
            assert ctas <= (16 if units <= room else 8)
            larger += ctas > 8
    assert larger > 0


def test_room_changes_nothing_else(shapes):
    for (rows, experts, N, sms, room, gated, dbias), got in shapes.items():
        without = shapes[rows, experts, N, sms, 0, gated, dbias]
        assert got[0] == without[0] and got[3:] == without[3:]
        assert got == without or (dbias and without[2] == 8 and got[1:3] == (256, 16))


def test_shapes_that_the_kernel_takes(shapes):
    for (rows, experts, N, sms, room, gated, dbias), (tx, threads, ctas, blocks, units) in shapes.items():
        assert threads in (256, 512) and tx in (4, 8, 16, 32, 64) and ctas >= 1 and ctas & (ctas - 1) == 0
        assert (blocks - 1) * 8 * tx < N <= blocks * 8 * tx and units == experts * blocks
        assert (2 if gated else 1) * (threads + tx) * 8 * 4 <= 48 * 1024   # (shared memory that needs no leave)
    assert shapes[16384, 1, 512, 152, 16, 0, 1] == (4, 256, 16, 16, 16)
    assert shapes[16384, 1, 512, 152, 0, 0, 1] == (4, 512, 8, 16, 16)
    assert shapes[16384, 1, 8192, 152, 16, 0, 1] == (8, 512, 2, 128, 128)
