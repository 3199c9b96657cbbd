"""The tile that a grouped product takes, on the CPU: the rule's ranges, each
tile reached, bad paths and shapes refused."""
import pytest

import block_scaled_precision_02_amd as q

I8, F8, MX8, MX4, BLOCK = range(5)


@pytest.mark.parametrize("path", [I8, F8, MX8, MX4, BLOCK])
def test_ranges(path):
    tall, most = (10, 448) if path == BLOCK else (5, 96)
    t = lambda rows, experts, N: q.select_grouped_tile(path, rows, experts, N)  # noqa: E731
    assert t(1, 1, 1) == 8 and t(16, 64, 512) == 8                      # few columns: the small-M kernel
    assert t(8, 64, 2048) == 16 and t(64, 16, 2112) == 16               # few workgroups, few rows: the stream
    assert t(40, 8, 4096) == 7                                          # more rows: 128x128
    assert t(128, 128, 4096) == 17 and t(1024, 64, 4096) == 17          # enough workgroups: 64-row panels
    assert t(1025, 64, 4096) == 18 and t(most * 64, 64, 4096) == 18     # above 16 rows an expert: 128x256
    assert t(17 * 16, 16, 3329) == 18 and t(17 * 16, 16, 3328) == 7     # where its workgroups nearly fill the chip: 16 x 14, 16 x 13
    assert t(most * 16, 16, 200) == 7
    assert t(most * 64 + 1, 64, 4096) == tall
    assert t(8192, 1, 4096) == tall


@pytest.mark.parametrize("args", [(-1, 8, 8, 64), (5, 8, 8, 64), (0, 0, 8, 64), (0, -3, 8, 64), (0, 1 << 30, 8, 64),
                                  (0, 8, 0, 64), (0, 8, 1025, 64), (0, 8, 8, 0), (0, 8, 8, 1 << 31)])
def test_refusals(args):
    assert q.select_grouped_tile(*args) == -1
