"""Runs the router, the few-token layer and the MXFP4 expert path some times each, for a profiler:

    rocprofv3 --kernel-trace -f csv -d DIR -o t -- python3 profiles/trace_operators.py

`python3 profiles/trace_operators.py DIR` then prints the table of operators.md.
"""
import csv
import glob
import os
import re
import statistics
import sys

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

CALLS = 20
CASES = ["Router, 1 token, E=32, top_k=8, fp32", "Router, 32768 tokens, E=256, top_k=8, bf16",
         "Few-token layer, M=1 K=7168 E=32 top_k=8 I=2048", "Few-token layer, M=5 K=4096 E=64 top_k=6 I=1408",
         "Few-token layer, M=16 K=7168 E=32 top_k=8 I=2048"]
CASES += [f"MXFP4 layer, M={M} K=7168 E=32 top_k=8 I=2048" for M in (1, 128, 512, 2048)]
CASES += ["MXFP4 layer, M=4096 K=4096 E=64 top_k=6 I=1408, Zipf(1.2) routing, 16 experts empty"]


def run():
    import torch
    from moe_expert_ffn_amd import megamoe as MM

    def rand(*shape, dtype=torch.float32):
        return torch.randn(shape, device="cuda", generator=gen).to(dtype)

    gen = torch.Generator(device="cuda").manual_seed(0)
    for M, E, dtype in ((1, 32, torch.float32), (32768, 256, torch.bfloat16)):
        logits, d = rand(M, E, dtype=dtype), MM.dims(M, 128, E, 8, 128)
        ids = torch.empty((M, 8), dtype=torch.int32, device="cuda")
        probs = torch.empty((M, 8), device="cuda")
        for _ in range(CALLS):
            MM.megamoe_route(d, logits, ids, probs)

    for M, K, E, top_k, I in ((1, 7168, 32, 8, 2048), (5, 4096, 64, 6, 1408), (16, 7168, 32, 8, 2048)):
        moe = MM.MegaMoE(M, K, E, top_k, I)
        for w in (moe.w1p, moe.w2p):
            w.random_(-127, 128, generator=gen)
        moe.scale1 = torch.full((E, 2 * I), 1e-3, device="cuda")
        moe.scale2 = torch.full((E, K), 1e-3, device="cuda")
        ids, probs = moe.route(rand(M, E))
        x = rand(M, K, dtype=torch.float16)
        for _ in range(CALLS):
            moe.forward_few(x, ids, probs)

    for M, K, E, top_k, I, routing in ((1, 7168, 32, 8, 2048, "uniform"), (128, 7168, 32, 8, 2048, "uniform"),
                                       (512, 7168, 32, 8, 2048, "uniform"), (2048, 7168, 32, 8, 2048, "uniform"),
                                       (4096, 4096, 64, 6, 1408, "zipf_empty")):
        moe = MM.MegaMoEMXFP4(M, K, E, top_k, I)
        moe.load_weights(rand(E, 2 * I, K, dtype=torch.bfloat16), rand(E, K, I, dtype=torch.bfloat16))
        logits = rand(M, E)
        if routing != "uniform":
            logits = -torch.log(-torch.log(torch.rand((M, E), device="cuda", generator=gen)))
            logits -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda"))
            logits[:, 3 * E // 4:] = -float("inf")
        ids, probs = moe.route(logits)
        x = rand(M, K, dtype=torch.float16)
        for _ in range(CALLS):
            moe.forward(x, ids, probs)
        del moe
    torch.cuda.synchronize()


def table(folder):
    titles = iter(CASES)
    cases, before = [], None
    for f in glob.glob(folder + "/**/*kernel_trace.csv", recursive=True):
        for r in sorted(csv.DictReader(open(f)), key=lambda r: int(r["Start_Timestamp"])):
            m = re.search(r"(?:megamoe::|_ZN7megamoe\d+)([a-z0-9_]+_kernel(?:<[^>]*>)?)", r["Kernel_Name"])
            if not m:
                continue
            key = (m.group(1), r["Grid_Size_X"], r["Grid_Size_Y"], r["Workgroup_Size_X"])
            if "route_topk" in key[0] and key != before:  # a case begins with its router
                cases.append((next(titles), {}))
            if cases:
                us = (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3
                cases[-1][1].setdefault(key, []).append(us)
            before = key
    for title, kernels in cases:
        print(f"\n{title}\n\n| kernel | workgroups | median us | min us |\n|---|---|---|---|")
        for (name, gx, gy, wx), us in kernels.items():
            if len(us) >= CALLS:
                print(f"| `{name}` | {int(gx) // int(wx)} x {gy} | {statistics.median(us):.1f} | {min(us):.1f} |")


if __name__ == "__main__":
    table(sys.argv[1]) if len(sys.argv) > 1 else run()
