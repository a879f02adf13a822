"""Times of the decoder-layer operators: the cases of perf/operators.py, or with
--more those of perf/more_operators.py, and any others of the same kinds.

    python examples/operator_times.py [name ...] [--case op=q8,M=512,N=8192,K=8192,epilogue=none ...] [--calls N]
    python examples/operator_times.py --more [name ...] [--case op=moe,T=16,E=8,H=4096,I=14336,top_k=2 ...] [--calls N]

Names select among the listed cases (none: all, or only those given with
--case).  For each case two times are printed, in
microseconds: of a call through the Python entry point, calls queued one after
the other, and of a call in a replayed graph, which leaves the host out.  Three
sets of operands and outputs take turns; what fits the last-level cache three
times over stays there.  GB/s and TFLOP/s are the case's bytes and operations, each counted
once, over the second time.  --calls makes that many calls of each case and
times nothing: for a profiler.
"""
import argparse
import importlib.util
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

DEFAULTS = {"norm": dict(stream="bf16", residual=True), "norm_q8": dict(stream="bf16", residual=True),
            "norm_backward": dict(stream="bf16", residual=True),
            "w4": dict(group=128, zeros=False, epilogue="none"), "q8": dict(epilogue="none")}
MORE_DEFAULTS = {"norm": DEFAULTS["norm"], "norm_backward": DEFAULTS["norm_backward"],
                 "lora": dict(rank=16, adapters=8, requests=8, epilogue="none"),
                 "moe": dict(renormalize=True, padded=0)}


def operators(file):
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", file))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    module.own = True
    return module


def parse_case(text):
    values = {}
    for part in text.split(","):
        key, _, value = part.partition("=")
        values[key] = int(value) if value.isdigit() else {"True": True, "False": False}.get(value, value)
    return dict(name=text, **values)


def median_us(fn, calls):
    """Median over 15 runs of `fn`, which makes `calls` calls, after a tenth of
    a second of them."""
    until = time.monotonic() + 0.1
    while time.monotonic() < until:
        fn()
        torch.cuda.synchronize()
    times = []
    for _ in range(15):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        fn()
        end.record()
        end.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / calls)
    return sorted(times)[7]


def measure(module, case):
    states = [module.prepare(case, seed) for seed in range(3)]
    calls = 3 if module.work(case)["flops"] > 1e11 else 24
    outputs = [None] * 3  # (three sets of them, too)

    def run():
        for i in range(calls):
            outputs[i % 3] = module.run(states[i % 3])

    run()
    torch.cuda.synchronize()
    eager = median_us(run, calls)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    graph.replay()
    torch.cuda.synchronize()
    return eager, median_us(graph.replay, calls)


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    parser.add_argument("names", nargs="*")
    parser.add_argument("--case", action="append", type=parse_case, default=[])
    parser.add_argument("--calls", type=int, default=0)
    parser.add_argument("--more", action="store_true")
    args = parser.parse_args(argv)
    defaults = MORE_DEFAULTS if args.more else DEFAULTS
    for case in args.case:
        if case.get("op") not in defaults:
            parser.error(f"op must be one of {', '.join(defaults)}")
    if not torch.cuda.is_available():
        raise SystemExit("these times need a GPU")
    module = operators("more_operators.py" if args.more else "operators.py")
    cases = [c for c in module.listed() if c["name"] in args.names or not (args.names or args.case)]
    cases += [{**defaults[c["op"]], **c} for c in args.case]
    for case in cases:
        if args.calls:
            state = module.prepare(case, 0)
            for _ in range(args.calls):
                module.run(state)
            torch.cuda.synchronize()
            print(case["name"], flush=True)
            continue
        eager, graph = measure(module, case)
        work = module.work(case)
        print(f"{case['name']:44s} call {eager:8.2f} us   in a graph {graph:8.2f} us   "
              f"{work['bytes'] / graph / 1e3:7.0f} GB/s {work['flops'] / graph / 1e6:8.1f} TFLOP/s", flush=True)


if __name__ == "__main__":
    main()
