"""Host-side model of the windows that moe_w4a16_token_logprobs puts aside while it reads a row.

Rows of values in no order have to fit the list that the kernel has for them (its length is read from the source), for
the most alternatives and rows longer than vocabularies are; else every such row would be read again."""
import os
import re

import numpy as np
import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a16_compact_expert_gb300", "csrc",
                      "logprobs.cu")


def rooms():
    """(windows, candidates) that a CTA of 128 threads or more has room for."""
    with open(SOURCE) as f:
        m = re.search(r"kWin = NT == 32 \? \d+ : (\d+), kCand = NT == 32 \? \d+ : (\d+);", f.read())
    return int(m.group(1)), int(m.group(2))


def put_aside(x, per_window, threads, k, unroll=4):
    """(windows put aside, values of the row that reach the last threshold)"""
    largest = x.reshape(-1, per_window).max(1)
    batches = -(-len(largest) // (unroll * threads))
    w = np.full(batches * unroll * threads, -np.inf, np.float32)
    w[:len(largest)] = largest
    w = w.reshape(batches, unroll, threads)
    best, bar, n = np.full(threads, -np.inf, np.float32), -np.inf, 0
    for b in range(batches):
        best = np.maximum(best, w[b].max(0))
        if b & (b + 1) == 0:
            bar = np.sort(best.reshape(64, -1).max(1))[-k]
        n += int((w[b] >= bar).sum())
    return n, int((x >= bar).sum())


@pytest.mark.parametrize("threads", [128, 512])
@pytest.mark.parametrize("per_window,V", [(4, 131072), (4, 200000), (4, 262144), (8, 151936), (8, 262144)])
def test_rows_in_no_order_fit(threads, per_window, V):
    win, cand = rooms()
    rng = np.random.default_rng(V + threads)
    for _ in range(25):
        x = (rng.standard_normal(V) * 2.5).astype(np.float32)
        n, reach = put_aside(x, per_window, threads, 32)
        assert 32 <= reach <= cand
        assert n <= win


def test_values_that_rise_to_the_last_threshold_do_not_fit_but_few_reach_it():
    """The rows of the GPU test for the second reading are what they are meant to be."""
    win, cand = rooms()
    for threads in (128, 512):
        n, reach = put_aside(rising(threads, 1), 4, threads, 20)
        assert n > win and 20 <= reach <= cand


def rising(threads, seed):
    """A row of FP32 that rises over the first 32 batches, with noise, and ends low."""
    V = 33 * 16 * threads
    x = np.arange(V, dtype=np.float32) / (16 * threads)
    x[V // 33 * 32:] = -4.0
    return x + np.random.default_rng(seed).standard_normal(V).astype(np.float32) * np.float32(0.05)
