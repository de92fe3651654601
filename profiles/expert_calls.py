"""The calls behind profiles/expert_products.md and their times: the cases of
perf/operators.py, and a few sizes that it does not list.

    python3 profiles/expert_calls.py times [--plain]      us of a call among others, and its floor
    python3 profiles/expert_calls.py calls N              N calls of every case, for the profiler
    python3 profiles/expert_calls.py table N TRACE PMC..  the markdown table, from the profiler's folders

`table` is given the folders that rocprofv3 wrote for `calls N` (one kernel trace, and counter
runs). It takes kernels in the order of their starts, so it needs the same N.
"""
import collections
import csv
import glob
import os
import re
import statistics
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

# What this card's own streams reach (bench.py's ceiling: read, write) in bytes/us, and the
# fastest large dense products of the library in operations/us.
READ, WRITE = 7.25e6, 7.00e6
RATE = {"bf16": 1635e6, "int8": 2454e6, "f32": 154e6}


def _layer(name, op, dtype, R, E, K, S, B, n_in, n_out, transposed):
    return {"name": name, "op": op, "dtype": dtype, "R": R, "E": E, "K": K, "S": S, "B": B, "n_in": n_in,
            "n_out": n_out, "transposed": transposed, "skew": 0.0}


def cases():
    import perf.operators as po
    return po, po.listed() + [
        _layer("short_f32", "matmul", "f32", 8, 128, 4, 256, 0, 2048, 1024, False),
        _layer("uniform_f32", "matmul", "f32", 8, 64, 8, 512, 8, 2048, 1024, False),
        _layer("int8_one_token", "int8", "bf16", 8, 64, 8, 1, 8, 2048, 1024, True),
        _layer("int8_uniform_f32", "int8", "f32", 8, 64, 8, 4096, 8, 2048, 1024, True),
    ]


def floor_us(po, case):
    """Least time of a call: its bytes at the streams' rates, or its operations."""
    import numpy as np
    if case["op"] == "clip":
        n = int(po._sizes(case).sum()) * (2 if case["dtype"] == "bf16" else 4)
        return 2 * n / READ + n / WRITE
    R, G, B, SK = case["R"], case["E"] // case["R"], case["B"], case["S"] * case["K"]
    n_in, n_out, es = case["n_in"], case["n_out"], 2 if case["dtype"] == "bf16" else 4
    lens = np.diff(po._table(case, 1)[0], axis=1)
    full = (lens > 0) & (np.arange(lens.shape[1]) < G + B)
    rows, segs = int(lens[full].sum()), int(full.sum())
    ops = 2.0 * rows * n_in * n_out
    if case["op"] == "wgrad":
        segs += R * G - int(full[:, :G].sum())
        return max(rows * (n_in + n_out) * es / READ + 4.0 * segs * n_in * n_out / WRITE,
                   ops / RATE[case["dtype"]])
    if case["op"] == "int8":
        quantised = R * SK * n_in * es / READ + R * SK * n_in / WRITE
        return quantised + max((rows * n_in + segs * n_in * n_out) / READ + rows * n_out * es / WRITE,
                               ops / RATE["int8"])
    return max((rows * n_in + segs * n_in * n_out) * es / READ + rows * n_out * es / WRITE,
               ops / RATE[case["dtype"]])


def times(plain):
    import torch
    po, cs = cases()
    po.own = not plain
    for c in cs:
        size = po.work(c)["bytes"]
        states = [po.prepare(c, s) for s in range(1, 2 if size > 2e9 else 4)]  # not from the caches
        n = 3 if plain else 12 if size > 1e9 else 300
        seen = []
        for _ in range(3 if plain else 7):
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            for i in range(n):
                po.run(states[i % len(states)])
            torch.cuda.synchronize()
            seen.append((time.perf_counter() - t0) / n * 1e6)
        print(f"{c['name']:20s} {statistics.median(seen):10.1f} us   floor {floor_us(po, c):8.1f} us", flush=True)
        del states


def calls(n):
    import torch
    po, cs = cases()
    po.own = True
    for c in cs:
        state = po.prepare(c, 1)
        for _ in range(n):
            po.run(state)
        torch.cuda.synchronize()
        print(c["name"], flush=True)
        del state


KERNELS = r"k_(matmul|wgrad|quantize|sumsq|join|clip)\b"


def _by_case(folder, what, cs, n):
    """(case, kernel) -> launches, each a dict of its counters and its duration."""
    launches = collections.OrderedDict()
    for path in sorted(glob.glob(folder + f"/**/*{what}.csv", recursive=True)):
        with open(path) as f:
            for r in csv.DictReader(f):
                if re.search(KERNELS, r["Kernel_Name"]):
                    e = launches.setdefault(int(r["Dispatch_Id"]), {"kernel": r["Kernel_Name"]})
                    e["at"] = int(r["Start_Timestamp"])
                    e["us"] = (int(r["End_Timestamp"]) - e["at"]) / 1e3
                    if "Counter_Name" in r:
                        e[r["Counter_Name"]] = float(r["Counter_Value"])
    order, at = sorted(launches.values(), key=lambda e: e["at"]), 0
    out = collections.OrderedDict()
    for c in cs:
        each = {"int8": 2, "clip": 3}.get(c["op"], 1)
        for e in order[at:at + n * each]:
            tile = re.search(r"Product<\d+, \w+, \w+, (\d+), (\d+)", e["kernel"])
            name = re.search(KERNELS, e["kernel"]).group(0) + (" %sx%s" % tile.groups() if tile else "")
            out.setdefault((c["name"], name), []).append(e)
        at += n * each
    assert at == len(order), f"{len(order)} launches, {at} expected"
    return out


def table(n, trace, counters):
    _, cs = cases()
    rows = _by_case(trace, "kernel_trace", cs, n)
    seen = collections.defaultdict(dict)
    for folder in counters:
        for key, launches in _by_case(folder, "counter_collection", cs, n).items():
            for counter in launches[0]:
                if counter not in ("kernel", "at"):
                    name = counter if counter != "us" else "us " + str(len(seen[key]))
                    seen[key][name] = statistics.median(e[counter] for e in launches[n // 2:])
                    if counter == "GRBM_GUI_ACTIVE":  # cycles, summed over 8 XCDs
                        seen[key]["GHz"] = statistics.median(e[counter] / 8 / e["us"] / 1e3
                                                             for e in launches[n // 2:])
    print("| call | kernel (tile) | least us | median us | GHz | matrix busy | LDS conflicts | read MB | written MB |")
    print("|---|---|---|---|---|---|---|---|---|")
    for (case, kernel), launches in rows.items():
        us = [e["us"] for e in launches[n // 2:]]
        c = seen[case, kernel]
        busy = c["SQ_VALU_MFMA_BUSY_CYCLES"] / (c["GRBM_GUI_ACTIVE"] / 8 * 256 * 4)
        # a launch's own cycles count before and after it too, which tells in short ones
        clock = f"{c['GHz']:.2f}" if statistics.median(us) > 200 else "-"
        print(f"| {case} | {kernel} | {min(us):.4g} | {statistics.median(us):.4g} | {clock} | {busy:.0%} | "
              f"{c['SQ_LDS_BANK_CONFLICT'] / max(1, c['SQ_LDS_IDX_ACTIVE']):.0%} | "
              f"{2 * c['FETCH_SIZE'] * 1024 / 1e6:.4g} | {c['WRITE_SIZE'] * 1024 / 1e6:.4g} |")


if __name__ == "__main__":
    if sys.argv[1:2] == ["times"]:
        times("--plain" in sys.argv)
    elif sys.argv[1:2] == ["calls"]:
        calls(int(sys.argv[2]))
    elif sys.argv[1:2] == ["table"]:
        table(int(sys.argv[2]), sys.argv[3], sys.argv[4:])
    else:
        sys.exit(__doc__)
