"""Calls of the 4-bit layer, the norms and the gated residuals in a loop, for a
profiler around it. Measurement infrastructure, not a test.

    rocprofv3 --kernel-trace --stats -d OUT -o r --output-format csv -- \\
        python3 tests/probes/operator_loop.py NAME[,NAME...] CALLS

NAME: a case of perf/operators.py, "quant_rows_fp32" (the fp32 form of
"quant_ffn_rows") or "all". Each case's call is made CALLS times over three
sets of inputs in turn, the weights and layers of each set made before.
"""
from __future__ import annotations

import importlib.util
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, ROOT)


def main(names: str, calls: str) -> int:
    import torch
    if not torch.cuda.is_available():
        print("no GPU", file=sys.stderr)
        return 2
    spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
    cases = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(cases)
    cases.own = True
    wanted = names.split(",")
    extra = cases.quant_case(8192, 12288, "float32", name="quant_rows_fp32")
    for case in cases.listed() + [extra]:
        if wanted != ["all"] and case["name"] not in wanted:
            continue
        sets = [cases.prepare(case, seed) for seed in range(3)]
        torch.cuda.synchronize()
        for i in range(int(calls)):
            cases.run(sets[i % 3])
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del sets
    return 0


if __name__ == "__main__":
    sys.exit(main(*sys.argv[1:3]))
