"""The loop that the profiles of speculative decoding with drafted trees were
taken from: every case that perf/operators.py lists, prepared with
prepare(case, 3) and run a given number of times by the library's calls.

    rocprofv3 --kernel-trace --stats --output-format csv -d out -o k -- python3 profiles/tree_speculation_loop.py 20

Prints each case with the bytes that these very inputs cannot do without (a
sequence without nodes, or with an empty path, needs none), which work(case)
gives as an average over ragged counts, empty paths included."""
import importlib.util
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
spec = importlib.util.spec_from_file_location("operators", os.path.join(ROOT, "perf", "operators.py"))
ops = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ops)


def bytes_of(case, state):
    counts = state.get("n_path" if case["op"] == "tree_commit" else "n_node")
    if counts is None or case["op"] == "tree_accept":
        return ops.work(case)["bytes"]
    B, H, e, D = case["B"], case["H"], 4 if case["dtype"] == "f32" else 2, 128
    some, tokens = int((counts > 0).sum()), int(counts.sum())
    if case["op"] == "tree_prologue":
        return tokens * H * (8 * D + 2) * e + some * 9 * H * D * e + 3 * H * D * 20
    if case["op"] == "tree_decode":
        return some * H * D * D * 4 + tokens * H * (5 * D + 1) * e
    return some * H * D * D * 8 + tokens * H * (3 * D + 1) * e + (some * 9 * H * D * e * 2 if case["conv"] else 0)


if __name__ == "__main__":
    ops.own = True
    for case in ops.listed():
        state = ops.prepare(case, 3)
        need = bytes_of(case, state)
        torch.cuda.synchronize()
        for _ in range(int(sys.argv[1])):
            ops.run(state)
        torch.cuda.synchronize()
        print(f"{case['name']}: {need} bytes", flush=True)
        del state
        torch.cuda.empty_cache()
