"""Every launch of the norm in blocks of 128, enumerated on the CPU from the rules in its source: threads within the
kernel's bound, every window of the longest row covered, and the block maxima of a CTA's rows within their array."""
import os
import re

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_compact_expert_gb300", "csrc",
                      "norm.cu")


def rules():
    with open(SOURCE) as f:
        s = f.read()
    tops, row_threads = map(int, re.search(r"constexpr int kTops = (\d+), kRowThreads = (\d+);", s).groups())
    lines = re.findall(r"(?:if \(windows <= (\d+)\) )?return launch_(rows|stream)<E, A, (\d+), (\d+), BLK>", s)
    return tops, row_threads, [(int(limit or 1 << 30), kind, int(v), int(mt)) for limit, kind, v, mt in lines]


def threads(windows, v):
    nt = -(-windows // v)
    if nt > 32:
        return -(-nt // 32) * 32
    return 1 << (nt - 1).bit_length()


def test_block_maxima_fit():
    tops, row_threads, lines = rules()
    assert [k for _, k, _, _ in lines].count("rows") == 4 and [k for _, k, _, _ in lines].count("stream") == 5
    for kind, first in (("rows", 1), ("stream", 97)):
        steps = [r for r in lines if r[1] == kind]
        for windows in range(first, (16384 + 14) // 8 + 1):
            _, _, v, mt = next(r for r in steps if windows <= r[0])
            nt = threads(windows, v)
            rows = row_threads // nt if kind == "rows" and nt < row_threads else 1
            assert nt * rows <= max(mt, row_threads) and nt <= mt and v * nt >= windows
            assert rows * -(-v * nt // 16) <= tops, (kind, windows)
            if nt > 32:
                assert nt % 32 == 0   # whole warps: a block is the windows of 16 lanes
