"""Times the cases of perf/operators.py or perf/more_operators.py on the GPU.

    python perf/timing.py [--more] [--plain] [--only NAME,NAME] [--repeats 7] [--once]

For each case: microseconds of a pass (CUDA events around passes that follow one
another, the median of the repeats), the same from a CUDA graph of one pass over
each input set (the device's time: no host between the launches), the host's time
for issuing a pass, and the rates of the first from the case's own bytes and
operations. Passes take turns on input sets that together exceed L2. --more takes the
cases of perf/more_operators.py; --plain times the plain forms; --once makes two passes of each case and no timing (to profile).
"""
import argparse
import importlib.util
import os
import statistics
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
L2 = 129 << 20


def load(name):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, "perf", name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def between(f, passes):
    """Microseconds a pass of f(i), on the device's clock."""
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for i in range(passes):
        f(i)
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) * 1e3 / passes


def captured(run, states):
    """A graph of one pass over each state."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(states[0])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = [run(s) for s in states]
    return graph, kept


def measure(ops, case, repeats):
    sets = max(3, min(24, -(-2 * L2 // int(ops.work(case)["bytes"]))))
    states = [ops.prepare(case, seed) for seed in range(sets)]
    call = lambda i: ops.run(states[i % sets])  # noqa: E731
    between(call, 5)
    passes = max(5, min(300, int(20e3 / between(call, 3))))  # about 20 ms
    stream = statistics.median(between(call, passes) for _ in range(repeats))
    host = []
    for _ in range(repeats):
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(20):  # few enough for the launch queue
            call(i)
        host.append((time.perf_counter() - t) * 1e6 / 20)
        torch.cuda.synchronize()
    device = None
    if ops.own:
        graph, _kept = captured(ops.run, states)
        replay = lambda i: graph.replay()  # noqa: E731
        between(replay, 2)
        device = statistics.median(between(replay, max(2, passes // sets)) for _ in range(repeats)) / sets
    return stream, device, statistics.median(host)


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--more", action="store_true")
    p.add_argument("--plain", action="store_true")
    p.add_argument("--only", default="")
    p.add_argument("--repeats", type=int, default=7)
    p.add_argument("--once", action="store_true")
    a = p.parse_args()
    ops = load("more_operators" if a.more else "operators")
    ops.own = not a.plain
    only = a.only.split(",") if a.only else None
    cases = [c for c in ops.listed() if not only or c["name"] in only]
    if a.once:
        for case in cases:
            state = ops.prepare(case, 0)
            ops.run(state)
            ops.run(state)
            torch.cuda.synchronize()
        return
    print(f"{'case':20s} {'us':>9s} {'graph us':>9s} {'host us':>8s} {'GB/s':>7s} {'TFLOP/s':>8s}")
    for case in cases:
        us, device, host = measure(ops, case, a.repeats)
        w = ops.work(case)
        print(f"{case['name']:20s} {us:9.1f} {'-' if device is None else format(device, '.1f'):>9s} {host:8.1f} "
              f"{w['bytes'] / us / 1e3:7.0f} {w['flops'] / us / 1e6:8.1f}", flush=True)
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
