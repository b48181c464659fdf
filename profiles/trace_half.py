"""Runs the 16-bit experts, their gradients, the norms and the router's gradient some times each, for a profiler, as
trace_operators.py does for the router, the few-token layer and the MXFP4 experts:

    rocprofv3 --kernel-trace -f csv -d DIR -o t -- python3 profiles/trace_half.py
    rocprofv3 --pmc COUNTERS -f csv -d DIR2 -o c -- python3 profiles/trace_half.py

`python3 profiles/trace_half.py DIR` then prints the tables of times of half.md, and with
`counters DIR2 DIR3 ...` those of the counters of one or more runs.
"""
import os
import re
import sys

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import trace_operators as T  # noqa: E402

BIG, SKEWED = (7168, 32, 8, 2048), (4096, 64, 6, 1408)
DIMS = {BIG: "K=7168 E=32 top_k=8 I=2048", SKEWED: "K=4096 E=64 top_k=6 I=1408, Zipf(1.2) routing"}
RUNS = [("layer", M, BIG) for M in (1, 128, 512, 2048)] + [("layer", 4096, SKEWED)]
RUNS += [(op, 2048, BIG) for op in ("gmm1", "gmm2", "gmm1_dgrad", "gmm2_dgrad", "gmm1_wgrad", "gmm2_wgrad")]
RUNS += [(op, 4096, SKEWED) for op in ("gmm1", "gmm2", "gmm1_dgrad", "gmm2_dgrad", "gmm1_wgrad", "gmm2_wgrad")]
RUNS += [("rows", 2048, BIG), ("router", 32768, (128, 256, 8, 128))]
NAMES = {"layer": "Layer, 16-bit experts", "rows": "SwiGLU, norms and their gradients", "router": "Router's gradient"}
T.CASES = [f"{NAMES.get(op, 'megamoe_half_' + op)}, M={M} " + DIMS.get(dims, "E=256 top_k=8") + ", bf16"
           for op, M, dims in RUNS]


def run():
    import torch
    from moe_expert_ffn_amd import half as H, megamoe as MM

    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    gen = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, dtype=bf16, scale=1.0):
        out = torch.empty(shape, dtype=dtype, device="cuda")
        for part in out if out.dim() == 3 else (out,):
            part.copy_(torch.randn(part.shape, device="cuda", generator=gen) * scale)
        return out

    def empty(*shape, dtype=bf16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    for op, M, (K, E, top_k, I) in RUNS:
        d, R = MM.dims(M, K, E, top_k, I), M * top_k
        logits = rand(M, E, dtype=f32)
        if E == 64:  # popularity of rank^-1.2
            logits = -torch.log(-torch.log(torch.rand((M, E), device="cuda", generator=gen)))
            logits -= 1.2 * torch.log(torch.arange(1, E + 1, device="cuda"))
        moe = None
        if op != "router":
            moe = H.MegaMoEHalf(M, K, E, top_k, I)
            moe.load_weights(rand(E, 2 * I, K, scale=K ** -0.5), rand(E, K, I, scale=I ** -0.5))
        x = rand(M, K)
        torch.cumsum(logits[:1], 1)  # another kernel between the cases
        ids, probs = empty(M, top_k, dtype=i32), empty(M, top_k, dtype=f32)
        MM.megamoe_route(d, logits, ids, probs)
        if op == "layer":
            for _ in range(T.CALLS):
                moe.forward(x, ids, probs)
        elif op == "router":
            half, dprobs, dlogits = logits.to(bf16), rand(M, top_k, dtype=f32), empty(M, E)
            for _ in range(T.CALLS):
                H.megamoe_route_grad(d, half, ids, probs, dprobs, dlogits, renormalize=False)
        else:
            row_of, route, count, end = (empty(n, dtype=i32) for n in (R, R, E, E))
            H.megamoe_sort_routes(d, ids, row_of, route, count, end, moe.workspace)
            c, y, rows, dc = rand(R, 2 * I), rand(R, I), rand(R, K), rand(R, 2 * I)
            dw1, dw2 = empty(E, 2 * I, K), empty(E, K, I)
            if op == "rows":
                w, gate, ws = rand(K, dtype=f32), rand(M, 1), empty(H.megamoe_norm_grad_workspace_bytes(d), dtype=torch.uint8)
                stream, s, r, h = rand(M, K, dtype=f32), empty(M, K), empty(M, K, dtype=f32), empty(M, K)
                dr, dx, ds, dgate = rand(M, K, dtype=f32), empty(M, K, dtype=f32), empty(M, K), empty(M, 1)
                dprobs, dw = empty(M, top_k, dtype=f32), [empty(K, dtype=f32) for _ in range(2)]
            for _ in range(T.CALLS):
                if op == "gmm1":
                    H.megamoe_half_gmm1(d, x, route, end, moe.w1, c)
                elif op == "gmm2":
                    H.megamoe_half_gmm2(d, y, end, moe.w2, rows)
                elif op == "gmm1_dgrad":
                    H.megamoe_half_gmm1_dgrad(d, dc, end, moe.w1, rows)
                elif op == "gmm2_dgrad":
                    H.megamoe_half_gmm2_dgrad(d, x, route, end, moe.w2, y)
                elif op == "gmm1_wgrad":
                    H.megamoe_half_gmm1_wgrad(d, dc, x, route, end, dw1)
                elif op == "gmm2_wgrad":
                    H.megamoe_half_gmm2_wgrad(d, x, y, route, end, dw2)
                else:
                    H.megamoe_half_swiglu(d, c, route, end, y, probs=probs)
                    H.megamoe_half_swiglu_grad(d, c, y, route, row_of, end, dc, probs=probs,
                                               dprobs=dprobs)
                    H.megamoe_norm(d, stream, rows, row_of, w, gate, 1.0, w, s=s, r=r, h=h)
                    H.megamoe_norm_grad(d, r, ws, dr, rows, row_of, s, w, gate, 1.0, w, dx=dx, ds=ds,
                                        dw_after=dw[0], dw_before=dw[1], dgate=dgate)
            del c, y, rows, dc, dw1, dw2
        del moe
        torch.cuda.empty_cache()
    torch.cuda.synchronize()


def read(folder, what, rows=T.read):
    """The profiler's rows, the tile kernel's geometry by what it computes."""
    kinds = ("product", "rows' gradient", "weights' gradient")
    out = []
    for r in rows(folder, what):
        m = re.search(r"half_gmm_kernel(?:<megamoe::HgGeom<(\d), \d, (\w+)|INS_6HgGeomILi(\d)ELi\dELb(\d))", r["Kernel_Name"])
        if m:
            kind, swiglu = (v for v in m.groups() if v is not None)
            name = f"megamoe::half_gmm_kernel<{kinds[int(kind)]}{', SwiGLU' if swiglu in ('1', 'true') else ''}>"
            r = {**r, "Kernel_Name": name}
        out.append(r)
    return out


T.read = read

if __name__ == "__main__":
    if len(sys.argv) < 2:
        run()
    elif sys.argv[1] == "counters":
        T.counters(sys.argv[2:])
    else:
        T.table(sys.argv[1])
