"""Times the listed cases of a workload file of this folder on the package's kernels.

    python perf/timing.py operators|more_operators [NAME ...]

Three figures for each case, microseconds a call:

* call — one call after another through the public entry points, each on other inputs than the last;
* GPU — the same calls, replayed from a CUDA graph;
* hot — a call on the same inputs over and over, replayed from a CUDA graph: what fits stays in L2.

There are as many sets of inputs as it takes to read and write three times the L2 between two uses of
one, up to 64 (calls that small stay in L2 all the same). CUDA events, the median of seven rounds.
"""
import importlib
import os
import statistics
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def timed(call, count):
    """Microseconds of one of the `count` calls that call() makes."""
    rounds = []
    for _ in range(3 + 7):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda.synchronize()
        start.record()
        call()
        end.record()
        torch.cuda.synchronize()
        rounds.append(start.elapsed_time(end) * 1e3 / count)
    return statistics.median(rounds[3:])


def captured(calls):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in calls:
            call()
    return graph


def main(module, names):
    cases = importlib.import_module("perf." + module)
    cases.own = True
    l2 = torch.cuda.get_device_properties(0).L2_cache_size
    print(f"{'':32} {'call':>9} {'GPU':>9} {'hot':>9}")
    for case in cases.listed():
        if names and case["name"] not in names:
            continue
        sets = int(max(2, min(64, 3 * l2 // cases.work(case)["bytes"] + 1)))
        states = [cases.prepare(case, seed) for seed in range(sets)]
        calls = [lambda state=state: cases.run(state) for state in states] * (-(-32 // sets))
        for call in calls[:sets]:
            call()
        torch.cuda.synchronize()
        graphs = [captured(calls), captured(calls[:1] * 32)]
        figures = [timed(lambda: [call() for call in calls], len(calls)), timed(graphs[0].replay, len(calls)),
                   timed(graphs[1].replay, 32)]
        print(f"{case['name']:32} " + " ".join(f"{f:9.2f}" for f in figures), flush=True)
        del states, calls, graphs
        torch.cuda.empty_cache()


if __name__ == "__main__":
    if len(sys.argv) < 2:
        sys.exit(__doc__)
    main(sys.argv[1], sys.argv[2:])
