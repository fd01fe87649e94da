"""The loop that the profiles of the 8-bit state cache and of sampling were taken
from: every case that perf/more_operators.py lists, prepared with
prepare(case, 3) and run a given number of times by the library's calls.

    rocprofv3 --kernel-trace --stats --output-format csv -d out -o k -- python3 profiles/cache_sampling_loop.py 20

A store's and a fold's result is not read back (that file's run() does so, to
compare values).  Prints each case with the bytes that these very inputs cannot do
without; a window's are those of the tokens that it holds, and a page that several
requests name counts once."""
import importlib.util
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
ops = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ops)
D = 128


def bytes_of(case, state):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "sample":
        return case["R"] * case["V"] * e * (2 if case["probs"] else 1) + case["R"] * 24
    H, packed = case["H"], D * D + 4 * D
    n_win, page = state.get("n_win"), state.get("page")
    busy = case["B"] if page is None else int((page >= 0).sum())
    tokens = 0 if n_win is None else int(n_win.clamp(min=0).sum())
    if case["op"] == "cache_store":
        return busy * H * (4 * D * D + packed)
    if case["op"] == "cache_load":
        pages = busy if page is None else int(page[page >= 0].unique().numel())
        return H * (pages * packed + busy * 4 * D * D + tokens * 3 * D * e)
    if case["op"] == "cache_fold":
        return H * (int((n_win > 0).sum()) * 2 * packed + tokens * 3 * D * e)
    # q, k, v, log alpha and o, beta, and the token's three rows
    return H * (int((n_win >= 0).sum()) * (packed + (8 * D + 1) * e) + tokens * 3 * D * e)


if __name__ == "__main__":
    ops.own = True
    ops._values = lambda codes, scale: codes
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
