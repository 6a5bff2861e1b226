"""Times of the expert-layer operators, through the package's own calls.

    python examples/time_expert_layers.py [--only TEXT]

The cases are those that perf/operators.py lists.  Calls go out one behind the
other, as in a model, on several sets of inputs in turn, so that together they
are larger than the L2 where their size allows; a call's time is that of the
sequence, from events around it, by its calls.  Beside it: the bytes and
operations that the call cannot do without, and the rates that these make.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mxfp4_gb300 as mx
from perf import operators

L2 = 130e6


def time_calls(states, seconds=0.5):
    """Microseconds of a call, the middle one of three sequences (long ones: the
    board's power holds the large products' clocks after some 0.1 s)."""
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))

    def sequence(rounds):
        start.record()
        for _ in range(rounds):
            for s in states:
                operators.run(s)
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) * 1e3 / (rounds * len(states))

    sequence(3)
    rounds = max(3, int(seconds * 1e6 / sequence(3) / len(states)))
    return sorted(sequence(rounds) for _ in range(3))[1]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--only", default="", help="cases whose name has this in it")
    a = ap.parse_args()
    operators.own = True
    for case in operators.listed():
        if a.only not in case["name"]:
            continue
        work = operators.work(case)
        sets = int(min(16, max(2, 1 + 2 * L2 // work["bytes"])))
        us = time_calls([operators.prepare(case, seed) for seed in range(sets)])
        print(f"{case['name']:18} {us:8.1f} us   {work['bytes'] / 1e6:8.2f} MB, {work['bytes'] / us / 1e6:5.2f} TB/s"
              f"   {work['flops'] / 1e9:7.2f} GFLOP, {work['flops'] / us / 1e6:7.1f} TFLOP/s   ({sets} sets of inputs)", flush=True)
        torch.cuda.empty_cache()
    assert mx.mxfp4_device_status() == 0


if __name__ == "__main__":
    main()
