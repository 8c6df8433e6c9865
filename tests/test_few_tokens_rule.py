"""Which kernels take 17 to 64 tokens of the 4-bit product with its epilogue: those that were the
faster by a tenth or more where both were measured.  Host logic only (csrc/linear_plan.h)."""
from __future__ import annotations

from host_forms_util import ask, build

# (tokens, d_out, d_in, group): us by tiles, us by the kernels for few tokens
MEASURED = {
    (64, 5120, 5120, 32): (23.4, 34.7), (64, 5120, 5120, 64): (22.5, 29.9), (64, 11008, 4096, 32): (27.2, 51.0),
    (64, 9216, 4096, 64): (24.9, 30.3), (64, 11008, 4096, 64): (26.1, 30.5), (64, 4096, 4096, 128): (18.7, 16.1),
    (64, 4096, 4096, -1): (17.7, 14.4), (64, 8192, 8192, -1): (25.5, 30.7), (64, 8192, 8192, 32): (32.7, 46.2),
    (48, 4096, 4096, 32): (18.4, 14.7), (48, 22016, 4096, 32): (39.8, 53.7), (48, 11008, 4096, 64): (24.8, 20.5),
    (33, 8192, 8192, 32): (28.5, 34.1), (33, 4096, 11008, 128): (26.7, 21.9), (33, 22016, 4096, 128): (35.4, 29.7),
    (33, 8192, 8192, -1): (22.6, 26.1), (48, 8192, 4096, -1): (19.9, 16.2), (32, 4096, 11008, 32): (25.4, 20.2),
    (32, 8192, 8192, 64): (23.5, 19.2), (32, 8192, 8192, 128): (23.2, 18.2), (17, 11008, 4096, -1): (16.4, 12.7),
}


def test_the_faster_kernels_are_taken(tmp_path):
    cases = [(m, n, k, g, 0) for m, n, k, g in MEASURED]
    for case, (tiles, few), line in zip(cases, MEASURED.values(), ask(build(tmp_path), cases)):
        assert line.split()[0] == ("vec" if few < tiles else "tiles"), (case, tiles, few, line)


def test_one_to_sixteen_tokens_and_many(tmp_path):
    cases = [(m, n, 4096, g, 0) for m in (1, 2, 16, 65, 1000) for n in (64, 57344) for g in (32, 64, 128, -1)]
    for (m, *_), line in zip(cases, ask(build(tmp_path), cases)):
        assert line.split()[0] == ("dot" if m == 1 else "vec" if m <= 16 else "tiles")
