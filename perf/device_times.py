"""Device time of the paged key-value cache operators, without the host's share.

    python perf/device_times.py                                 the listed cases
    python perf/device_times.py attend_long evict_small         some of them
    python perf/device_times.py attend:seqs=100,q_heads=32,tokens=200,cache=e4m3
                                                                any case, by the fields of operators._case

Twelve calls on three states in turn are captured into a CUDA graph and replayed; the best of five replays counts.
Beside it, the bytes that the case cannot do without and the rate that they move at.  What moves less than the L2
cache holds (about 40 MB in three states) is read from there.
"""
import os
import sys

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]

import torch  # noqa: E402

import operators  # noqa: E402


def case_of(text):
    """A listed case by its name, or one from op:field=value,.."""
    op, colon, fields = text.partition(":")
    if not colon:
        return next(c for c in operators.listed() if c["name"] == text)
    got = {}
    for f in filter(None, fields.split(",")):
        k, v = f.split("=")
        got[k] = v == "True" if v in ("True", "False") else int(v) if v.lstrip("-").isdigit() else v
    return operators._case(op, name=text, **got)


def device_us(case, calls=12, states=3, replays=5):
    held = [operators.prepare(case, seed) for seed in range(states)]
    for s in held:
        operators.run(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(calls):
            operators.run(held[i % states])
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    best = float("inf")
    for i in range(3 + replays):
        start.record()
        graph.replay()
        end.record()
        end.synchronize()
        if i >= 3:
            best = min(best, start.elapsed_time(end) / calls * 1e3)
    return best


def main():
    operators.own = True
    for case in [case_of(x) for x in sys.argv[1:]] or operators.listed():
        us, least = device_us(case), operators.work(case)["bytes"]
        print("%-40s %9.2f us  %9.1f MB  %7.1f GB/s" % (case["name"], us, least / 1e6, least / us / 1e3), flush=True)


if __name__ == "__main__":
    main()
