"""The calls behind layer_operators.md: every listed case of perf/more_operators.py, N times.

  python3 profiles/layer_calls.py calls N            makes them (under rocprofv3)
  python3 profiles/layer_calls.py table N TRACE_DIR COUNTER_DIR...   prints the table
  python3 profiles/layer_calls.py lengths            times the row kernels at every length of row
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


def lengths():
    """TB/s of the bytes that a call must move, ten calls together, 134 MB each operand."""
    import torch
    import token_dispatch_amd as td

    def timed(call, moved):
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        for _ in range(3):
            call()
        begin.record()
        for _ in range(10):
            call()
        end.record()
        torch.cuda.synchronize()
        return "%.2f" % (moved * 10 / begin.elapsed_time(end) / 1e9)

    for dtype in (torch.bfloat16, torch.float32):
        es = torch.finfo(dtype).bits // 8
        for cols in (32, 64, 128, 256, 512, 1024, 2048, 4096, 5792, 7168, 12288, 16384):
            rows = (1 << 27) // es // cols
            x, r, s, o = (torch.randn(rows, cols, device="cuda").to(dtype) for _ in range(4))
            g, gg, work = s[0].clone(), torch.empty(cols, device="cuda"), td.new_norm_workspace(cols)
            inv, qs = (torch.ones(rows, device="cuda") for _ in range(2))
            q = torch.empty(rows, cols, device="cuda", dtype=torch.int8)
            q4 = torch.empty(rows, cols // 2, device="cuda", dtype=torch.uint8)
            s4 = torch.empty(rows, td.mx_scale_cols(cols), device="cuda", dtype=torch.uint8)
            n = rows * cols
            print("| %s %d |" % ("bf16" if es == 2 else "f32", cols), " | ".join((
                timed(lambda: td.moonep_rmsnorm(x, g, o, 1e-6, residual=r, sum_out=s), 4 * es * n),
                timed(lambda: td.moonep_rmsnorm_quant(x, g, q, qs, 1e-6, residual=r, sum_out=s), (3 * es + 1) * n),
                timed(lambda: td.moonep_rmsnorm_mx(x, g, q4, s4, 1e-6, residual=r, sum_out=s), (3 * es + .53) * n),
                timed(lambda: td.moonep_rmsnorm_backward(x, r, g, inv, o, gg, work, grad_sum=s), 4 * es * n),
                timed(lambda: td.moonep_swiglu(x, r, o), 3 * es * n),
                timed(lambda: td.moonep_swiglu_quant(x, r, q, qs), (2 * es + 1) * n),
                timed(lambda: td.moonep_swiglu_mx(x, r, q4, s4), (2 * es + .53) * n),
                timed(lambda: td.moonep_swiglu_backward(x, r, s, o, s), 5 * es * n),
                timed(lambda: td.moonep_quantize_rows_mx(x, q4, s4), (es + .53) * n))), "|", flush=True)


if __name__ == "__main__":
    if sys.argv[1] == "calls":
        calls(int(sys.argv[2]))
    elif sys.argv[1] == "lengths":
        lengths()
    else:
        table(int(sys.argv[2]), *sys.argv[3:])
