"""The calls behind layer_operators.md: every listed case of perf/more_operators.py, N times.

  python3 profiles/layer_calls.py calls N            makes them (under rocprofv3)
  python3 profiles/layer_calls.py table N TRACE_DIR COUNTER_DIR...   prints the table
"""
import csv
import glob
import importlib.util
import os
import re
import statistics
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


def cases():
    spec = importlib.util.spec_from_file_location("cases", os.path.join(ROOT, "perf", "more_operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.own = True
    return mod


def calls(n):
    import torch
    mod = cases()
    for case in mod.listed():
        state = mod.prepare(case, 1)
        for _ in range(n):
            mod.run(state)
        torch.cuda.synchronize()
        print(case["name"], flush=True)
        del state
        torch.cuda.empty_cache()


def rows_of(path, pattern):
    files = glob.glob(os.path.join(path, "**", pattern), recursive=True)
    rows = [r for f in files for r in csv.DictReader(open(f)) if "moonep" in r["Kernel_Name"]]
    return sorted(rows, key=lambda r: int(r.get("Start_Timestamp") or r["Dispatch_Id"]))


def short(name):
    name = re.sub(r"moonep::|\(anonymous namespace\)::|void ", "", name)
    return re.sub(r"ScaledProduct<([^>]*)>, ", "", name.split("(")[0])


def table(n, trace, *counters):
    mod, out = cases(), []
    launches = rows_of(trace, "*kernel_trace.csv")
    count = {}
    for path in counters:
        seen = {}
        for r in rows_of(path, "*counter_collection.csv"):
            seen.setdefault(r["Counter_Name"], []).append(float(r["Counter_Value"]))
        count.update(seen)
    at = 0
    for case in mod.listed():
        # the launches of one call: until the first kernel's name comes again
        names = [r["Kernel_Name"] + r["Grid_Size_X"] for r in launches[at:at + 8]]
        each = next(k for k in range(1, 9) if k == len(names) or names[k] == names[0])
        for j in range(each):
            pick = range(at + j + each * (n // 2), at + each * n, each)
            us = [(int(launches[i]["End_Timestamp"]) - int(launches[i]["Start_Timestamp"])) / 1e3 for i in pick]
            c = {k: statistics.median(v[i] for i in pick) for k, v in count.items()}
            busy = 100 * c.get("SQ_VALU_MFMA_BUSY_CYCLES", 0) / (c.get("GRBM_GUI_ACTIVE", 1) / 8 * 1024)
            lds = 100 * c.get("SQ_LDS_BANK_CONFLICT", 0) / max(1, c.get("SQ_LDS_IDX_ACTIVE", 0))
            mid = statistics.median(us)
            read, written = 2 * 1024 * c.get("FETCH_SIZE", 0) / 1e6, 1024 * c.get("WRITE_SIZE", 0) / 1e6
            out.append("| %s | %s | %.4g | %.4g | %.0f%% | %.0f%% | %.4g | %.4g | %.3g |" % (
                case["name"], short(launches[at + j]["Kernel_Name"]), min(us), mid, busy, lds, read, written,
                (read + written) / mid))
        at += each * n
    print("| case | kernel | least us | median us | matrix busy | LDS conflicts | read MB | written MB | TB/s |")
    print("|---|---|---|---|---|---|---|---|---|")
    print("\n".join(out))


if __name__ == "__main__":
    if sys.argv[1] == "calls":
        calls(int(sys.argv[2]))
    else:
        table(int(sys.argv[2]), *sys.argv[3:])
