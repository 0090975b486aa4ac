"""Calls of the timed cases in a loop, for a profiler, and tables of what it wrote.

    rocprofv3 --kernel-trace --stats -d DIR -f csv -- python3 perf/loop.py run more_operators 120
    python3 perf/loop.py durations more_operators DIR
    rocprofv3 --pmc ... --kernel-trace -d DIR -f csv -- python3 perf/loop.py run more_operators 2
    python3 perf/loop.py counters more_operators DIR [DIR ...]

``run`` takes the listed cases of perf/<module>.py through the library, three
inputs in turn, with a kernel between two cases that no case launches; by that
the tables tell them apart.
"""
import collections
import csv
import glob
import importlib.util
import os
import re
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MARK = "BitwiseXorFunctor"


def cases(module):
    spec = importlib.util.spec_from_file_location(module, os.path.join(ROOT, "perf", module + ".py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def run(module, calls):
    import torch
    sys.path.insert(0, ROOT)
    m = cases(module)
    m.own = True
    mark = torch.zeros(64, dtype=torch.int32, device="cuda")
    for case in m.listed():
        states = [m.prepare(case, seed) for seed in range(3)]
        mark ^= 1
        for i in range(calls):
            m.run(states[i % 3])
        mark ^= 1
        torch.cuda.synchronize()
        print(case["name"], flush=True)


def rows(directory, kind):
    (at,) = glob.glob(os.path.join(directory, "**", f"*_{kind}.csv"), recursive=True)
    with open(at) as f:
        return list(csv.DictReader(f))


def by_case(module, dispatches):
    """(case, kernel, dispatch) of the library's kernels between a case's two marks."""
    names = [c["name"] for c in cases(module).listed()]
    marks = 0
    for d in dispatches:
        if MARK in d["Kernel_Name"]:
            marks += 1
        elif marks % 2 == 1 and "pq1" in d["Kernel_Name"]:
            kernel = re.sub(r"_ZN3pq112_GLOBAL__N_1\d\d", "", d["Kernel_Name"])
            yield names[marks // 2], re.search(r"([a-z]\w*_kernel)", kernel).group(1), d
    assert marks == 2 * len(names), f"{marks} marks of {len(names)} cases"


def durations(module, directory):
    """Durations of the last 20 launches of each kernel of a case."""
    trace = sorted(rows(directory, "kernel_trace"), key=lambda r: int(r["Start_Timestamp"]))
    times = collections.OrderedDict()
    for case, kernel, d in by_case(module, trace):
        key = (case, kernel)
        times.setdefault(key, []).append((int(d["End_Timestamp"]) - int(d["Start_Timestamp"])) / 1e3)
    print("| case | kernel | launches | p10 us | p50 us | p90 us |\n|---|---|---:|---:|---:|---:|")
    for (case, kernel), t in times.items():
        last = sorted(t[-20:])
        p = [last[int(q * (len(last) - 1) + 0.5)] for q in (0.1, 0.5, 0.9)]
        print(f"| {case} | `{kernel}` | {len(t)} | " + " | ".join(f"{x:.1f}" for x in p) + " |")


def counters(module, directories):
    """Counters of the last launch of each kernel of a case."""
    table = collections.OrderedDict()
    for directory in directories:
        dispatches = collections.OrderedDict()
        for r in sorted(rows(directory, "counter_collection"), key=lambda r: int(r["Dispatch_Id"])):
            d = dispatches.setdefault(r["Dispatch_Id"], {"Kernel_Name": r["Kernel_Name"]})
            d[r["Counter_Name"]] = float(r["Counter_Value"])
        for case, kernel, d in by_case(module, dispatches.values()):
            table.setdefault((case, kernel), {}).update(
                (k, v) for k, v in d.items() if k != "Kernel_Name")
    for (case, kernel), c in table.items():
        print(f"\n{case}, {kernel}")
        for name in sorted(c):
            print(f"  {name:28s} {c[name]:.0f}")
        busy = c["SQ_BUSY_CU_CYCLES"]
        print(f"  mfma_busy {c['SQ_VALU_MFMA_BUSY_CYCLES'] / 4 / busy:.3f}"
              f"  valu_active {c['SQ_ACTIVE_INST_VALU'] / busy:.3f}"
              f"  waiting {c['SQ_WAIT_ANY'] / c['SQ_WAVE_CYCLES']:.3f}")


if __name__ == "__main__":
    command, module = sys.argv[1:3]
    if command == "run":
        run(module, int(sys.argv[3]))
    elif command == "durations":
        durations(module, sys.argv[3])
    elif command == "counters":
        counters(module, sys.argv[3:])
    else:
        raise SystemExit(__doc__)
