"""Runs the router, the few-token layer and the MXFP4 expert path some times each, for a profiler:

    rocprofv3 --kernel-trace -f csv -d DIR -o t -- python3 profiles/trace_operators.py
    rocprofv3 --pmc COUNTERS -f csv -d DIR2 -o c -- python3 profiles/trace_operators.py

`python3 profiles/trace_operators.py DIR` then prints the tables of times of operators.md, and with
`counters DIR2 DIR3 ...` those of the counters of one or more runs.
"""
import collections
import csv
import glob
import os
import re
import statistics
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

CALLS = 20
CASES = ["Router, 1 token, E=32, top_k=8, fp32", "Router, 32768 tokens, E=256, top_k=8, bf16",
         "Router, the same with a bias and all experts' weights",
         "Few-token layer, M=1 K=7168 E=32 top_k=8 I=2048",
         "Few-token layer, M=5 K=4096 E=64 top_k=6 I=1408, Zipf(1.2) routing",
         "Few-token layer, M=16 K=7168 E=32 top_k=8 I=2048"]
CASES += ["MXFP4 rows, 128 x 7168 fp16 and back to bf16", "MXFP4 rows, 16384 x 2048 bf16 and back, 16211 of them valid"]
CASES += [f"MXFP4 layer, M={M} K=7168 E=32 top_k=8 I=2048" for M in (1, 128, 512, 2048)]
CASES += ["MXFP4 GMM1 alone (y in bf16), M=2048 K=7168 E=32 top_k=8 I=2048"]
CASES += ["MXFP4 layer, M=4096 K=4096 E=64 top_k=6 I=1408, Zipf(1.2) routing, 16 experts empty"]


def run():
    import torch
    from moe_expert_ffn_amd import megamoe as MM

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", generator=gen).to(dtype)

    def zipf(M, E, empty):
        """Logits whose top_k pick experts with a popularity of rank^-1.2, the last `empty` never."""
        logits = -torch.log(-torch.log(torch.rand((M, E), device="cuda", generator=gen)))
        logits -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda"))
        logits[:, E - empty:] = -float("inf")
        return logits

    gen = torch.Generator(device="cuda").manual_seed(0)
    for M, E, dtype, biased in ((1, 32, torch.float32, False), (32768, 256, torch.bfloat16, False),
                                (32768, 256, torch.bfloat16, True)):
        logits, d = rand(M, E, dtype=dtype), MM.dims(M, 128, E, 8, 128)
        bias = rand(E) * 0.1 if biased else None
        ids = torch.empty((M, 8), dtype=torch.int32, device="cuda")
        probs = torch.empty((M, 8), device="cuda")
        torch.cumsum(logits[:1].float(), 1)  # another kernel between the cases
        for _ in range(CALLS):
            MM.megamoe_route(d, logits, ids, probs, bias=bias, renormalize=not biased)

    for M, K, E, top_k, I, skewed in ((1, 7168, 32, 8, 2048, False), (5, 4096, 64, 6, 1408, True),
                                      (16, 7168, 32, 8, 2048, False)):
        moe = MM.MegaMoE(M, K, E, top_k, I)
        for w in (moe.w1p, moe.w2p):
            w.random_(-127, 128, generator=gen)
        moe.scale1 = torch.full((E, 2 * I), 1e-3, device="cuda")
        moe.scale2 = torch.full((E, K), 1e-3, device="cuda")
        ids, probs = moe.route(zipf(M, E, 0) if skewed else rand(M, E))
        x = rand(M, K, dtype=torch.float16)
        for _ in range(CALLS):
            moe.forward_few(x, ids, probs)

    for rows, cols, dtype, valid in ((128, 7168, torch.float16, 128), (16384, 2048, torch.bfloat16, 16211)):
        x, n = rand(rows, cols, dtype=dtype), torch.tensor([valid], dtype=torch.int32, device="cuda")
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device="cuda")
        scale = torch.empty((rows, cols // 32), dtype=torch.uint8, device="cuda")
        back = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
        MM.megamoe_route(MM.dims(1, 128, 32, 8, 128), rand(1, 32), torch.empty((1, 8), dtype=torch.int32, device="cuda"),
                         torch.empty((1, 8), device="cuda"))
        for _ in range(CALLS):
            MM.megamoe_mxfp4_quant(x, q, scale, valid_rows=n)
            MM.megamoe_mxfp4_dequant(q, scale, back, valid_rows=n)

    for M, K, E, top_k, I, skewed, alone in ((1, 7168, 32, 8, 2048, False, False), (128, 7168, 32, 8, 2048, False, False),
                                             (512, 7168, 32, 8, 2048, False, False), (2048, 7168, 32, 8, 2048, False, False),
                                             (2048, 7168, 32, 8, 2048, False, True), (4096, 4096, 64, 6, 1408, True, False)):
        moe = MM.MegaMoEMXFP4(M, K, E, top_k, I)
        moe.load_weights(rand(E, 2 * I, K, dtype=torch.bfloat16), rand(E, K, I, dtype=torch.bfloat16))
        ids, probs = moe.route(zipf(M, E, E // 4) if skewed else rand(M, E))
        x = rand(M, K, dtype=torch.float16)
        if not alone:
            for _ in range(CALLS):
                moe.forward(x, ids, probs)
        else:
            flat = ids.reshape(-1)
            order = torch.argsort(flat, stable=True).to(torch.int32)
            cumsum = torch.cumsum(torch.bincount(flat, minlength=E), 0).to(torch.int32)
            xq = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda")
            xs = torch.empty((M, K // 32), dtype=torch.uint8, device="cuda")
            y = torch.empty((M * top_k, I), dtype=torch.bfloat16, device="cuda")
            MM.megamoe_mxfp4_quant(x, xq, xs)
            for _ in range(CALLS):
                MM.megamoe_mxfp4_gmm1(moe.d, xq, xs, order, cumsum, moe.w1q, moe.w1s, y)
        del moe
    torch.cuda.synchronize()


def by_case(rows, order):
    """Rows of a profiler's csv -> [(title, {(kernel, grid...): rows})], a case from its router on."""
    titles, cases, before = iter(CASES), [], None
    for r in sorted(rows, key=lambda r: int(r[order])):
        m = re.search(r"(?:megamoe::|_ZN7megamoe\d+)([a-z0-9_]+_kernel(?:<[^>]*>)?)", r["Kernel_Name"])
        if not m:
            before = None if "route_topk" in (before or "") else before
            continue
        if "route_topk" in m.group(1) and "route_topk" not in (before or ""):
            cases.append((next(titles), {}))
        before = m.group(1)
        if cases:
            key = (m.group(1),) + tuple(r.get(c, "") for c in ("Grid_Size_X", "Grid_Size_Y", "Workgroup_Size_X"))
            cases[-1][1].setdefault(key, []).append(r)
    return cases


def read(folder, what):
    return [r for f in glob.glob(f"{folder}/**/*{what}.csv", recursive=True) for r in csv.DictReader(open(f))]


def table(folder):
    for title, kernels in by_case(read(folder, "kernel_trace"), "Start_Timestamp"):
        print(f"\n{title}\n\n| kernel | workgroups | median us | min us |\n|---|---|---|---|")
        for (name, gx, gy, wx), rows in kernels.items():
            us = [(int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3 for r in rows]
            if len(us) >= CALLS:
                print(f"| `{name}` | {int(gx) // int(wx)} x {gy} | {statistics.median(us):.1f} | {min(us):.1f} |")


def counters(folders):
    merged = collections.OrderedDict()  # (title, kernel) -> counter -> median over the dispatches
    for folder in folders:
        for title, kernels in by_case(read(folder, "counter_collection"), "Dispatch_Id"):
            for key, rows in kernels.items():
                values = collections.defaultdict(list)
                for r in rows:
                    values[r["Counter_Name"]].append(float(r["Counter_Value"]))
                    if r["Counter_Name"] == "GRBM_GUI_ACTIVE":  # summed over 8 XCDs
                        ns = int(r["End_Timestamp"]) - int(r["Start_Timestamp"])
                        values["ns"].append(ns)
                        values["GHz"].append(float(r["Counter_Value"]) / 8 / ns)
                if all(len(v) >= CALLS for v in values.values()):
                    merged.setdefault((title, key[0]), {}).update({n: statistics.median(v) for n, v in values.items()})
    title = None
    for (t, name), v in merged.items():
        if t != title:
            title = t
            print(f"\n{t}\n\n| kernel | GHz | MFMA busy | VALU active | LDS active | LDS conflicts | read MB | written MB |\n|---|---|---|---|---|---|---|---|")
        cycles = v["GRBM_GUI_ACTIVE"] / 8
        busy = [v["SQ_VALU_MFMA_BUSY_CYCLES"] / (1024 * cycles), v["SQ_ACTIVE_INST_VALU"] * 4 / (1024 * cycles),
                v["SQ_LDS_IDX_ACTIVE"] / (256 * cycles), v["SQ_LDS_BANK_CONFLICT"] / (256 * cycles)]
        clock = f"{v['GHz']:.2f}" if v["ns"] > 50e3 else ""  # the count takes in the dispatch of a short kernel
        print(f"| `{name}` | {clock} | " + " | ".join(f"{100 * b:.0f}%" for b in busy)
              + f" | {2 * v['FETCH_SIZE'] * 1024 / 1e6:.1f} | {v['WRITE_SIZE'] * 1024 / 1e6:.1f} |")


if __name__ == "__main__":
    if len(sys.argv) < 2:
        run()
    elif sys.argv[1] == "counters":
        counters(sys.argv[2:])
    else:
        table(sys.argv[1])
