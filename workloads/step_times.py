"""Times of the serving-step operators on this GPU: `python -m workloads.step_times [4-bit|8-bit] [name ...]`.

For each case of perf/operators.py (4-bit) and of perf/more_operators.py (8-bit), and for head counts that they do not
list, the time of a call among 20 in a captured graph, over two sets of inputs in turn (those of the large cases
exceed L2, those of the small ones stay in it), median of nine replays after two.  The decode cases are timed on a bf16
cache of the same lengths too, by the same method, with the group size that decode_auto_split_tokens picks.
"""
from __future__ import annotations

import statistics
import sys

import torch

import attention_attn_prefill_gb300 as attn
import perf.more_operators as more_ops
import perf.operators as ops

CALLS = 20
# query heads a KV head other than the listed 4 (d = 128) and 8 (d = 256), and the smallest head dim
FORMS = [dict(op="decode", name=f"decode {Hq}/{Hkv} d={d} N={N}", N=N, len_lo=lo, len_hi=hi, Hq=Hq, Hkv=Hkv, d=d)
         for N, lo, hi, Hq, Hkv, d in [
             (64, 512, 8192, 8, 8, 128), (64, 512, 8192, 40, 8, 128), (64, 512, 8192, 64, 8, 128),
             (64, 512, 8192, 64, 4, 128), (64, 8704, 8704, 32, 8, 64), (64, 8704, 8704, 64, 8, 64),
             (8, 6335, 122863, 8, 2, 256), (8, 6335, 122863, 2, 2, 256), (8, 6335, 122863, 32, 2, 256)]]


def graph_us(runs) -> float:
    """Microseconds of a call, `runs` taken in turn."""
    for run in runs:
        run()
    torch.cuda.synchronize()
    graph, keep = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for i in range(CALLS):
            keep = keep[-1:] + [runs[i % len(runs)]()]
    times = []
    for _ in range(11):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in "ab")
        start.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end) * 1e3 / CALLS)
    return statistics.median(times[2:])


def _bf16(state):
    """decode_paged on random bf16 pages of the same lengths and tables."""
    rec = state["cache"]
    shape = (rec.shape[0], ops.PAGE, state["Hkv"], state["d"])
    k, v = (torch.randn(shape, device="cuda", dtype=torch.bfloat16) for _ in "kv")
    tokens = attn.decode_auto_split_tokens(state["seq_lens"].cpu(), state["Hkv"], state["d"],
                                           state["block_table"].shape[1])
    return lambda: attn.decode_paged(state["q"], k, v, state["block_table"], state["seq_lens"], num_splits=0,
                                     split_tokens=tokens)


def main(names) -> None:
    kinds = {"4-bit": ops, "8-bit": more_ops}
    wanted = [x for x in names if x in kinds] or list(kinds)
    names = [x for x in names if x not in kinds]
    for kind in wanted:
        mod = kinds[kind]
        for case in mod.listed() + FORMS:
            if names and case["name"] not in names:
                continue
            mod.own = False
            states = [mod.prepare(case, seed) for seed in (1, 2)]
            mod.own = True
            us, work = graph_us([lambda s=s: mod.run(s) for s in states]), mod.work(case)
            line = (f"{kind} {case['name']:26s} {us:8.2f} us {work['bytes'] / us / 1e3:8.1f} GB/s"
                    f" {work['flops'] / us / 1e6:8.1f} TFLOP/s")
            if mod is ops and case["op"] == "decode" and case["d"] > 64:  # decode_paged takes head dims of 128 and 256
                line += f"   bf16 cache {graph_us([_bf16(s) for s in states]):8.2f} us"
            print(line, flush=True)
            del states


if __name__ == "__main__":
    main(sys.argv[1:])
