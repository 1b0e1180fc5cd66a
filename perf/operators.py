"""Cases and plain forms of the ragged expert products and of the orthogonalised update.

Four operators over E experts whose rows lie in expert-contiguous segments
[offsets[e], offsets[e+1]) of a row tensor, as moe_permute leaves them:

  gemm    y[r]  = x[r] W_e^T          x [M, K], W [E, N, K]  -> y  [M, N]
  dgrad   dx[r] = dy[r] W_e           dy [M, N]              -> dx [M, K]
  wgrad   dW_e  = dy_e^T x_e                                 -> dW [E, N, K] fp32
  ortho   U_b   = the Newton-Schulz iterate of g_b [B, M, N] -> U  [B, M, N] bf16
          X = g / ||g||_F, then `steps` times X <- a X + (b A + c A A) X with A = X X^T

With ``own`` false, run() computes them with elementary torch operations in 32 bits; with ``own``
true it calls this package's entry points.
"""
import functools
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)  # a, b, c of the quintic iteration
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ the cases
def _grouped(name, op, T, k, E, N, K, dtype, out="same", skew=0.0):
    return {"name": name, "op": op, "T": T, "k": k, "E": E, "N": N, "K": K, "dtype": dtype, "out": out, "skew": skew}


def _ortho(name, B, M, N, rows, dtype):
    return {"name": name, "op": "ortho", "B": B, "M": M, "N": N, "rows": rows, "dtype": dtype}


def listed():
    return [
        # one token of a decode loop through the first projection of its 4 experts
        _grouped("gemm_one_token", "gemm", 1, 4, 32, 5760, 2880, "bf16"),
        # a decode batch on a 32-expert layer with long rows: most experts get a few rows each
        _grouped("gemm_decode_64", "gemm", 64, 8, 32, 4096, 7168, "bf16"),
        # a prompt chunk with unbalanced experts
        _grouped("gemm_prefill", "gemm", 8192, 4, 32, 5760, 2880, "bf16", skew=0.5),
        # a small layer with sizes that divide by no tile, results kept in fp32 for a later sum
        _grouped("gemm_odd", "gemm", 777, 2, 8, 1000, 520, "fp16", out="fp32"),
        # the input gradient of a wide down projection in a training step
        _grouped("dgrad_train", "dgrad", 4096, 2, 8, 4096, 14336, "bf16"),
        # the same of a small model with odd sizes
        _grouped("dgrad_odd", "dgrad", 300, 3, 16, 712, 456, "fp16"),
        # weight gradients of square projections, about 1000 rows an expert
        _grouped("wgrad_train", "wgrad", 8192, 4, 32, 2880, 2880, "bf16", skew=0.5),
        # weight gradients of fine-grained experts: about 256 rows each, bound by writing dW
        _grouped("wgrad_fine", "wgrad", 1024, 8, 32, 4096, 7168, "bf16"),
        # a small model's, with empty and ragged experts
        _grouped("wgrad_odd", "wgrad", 500, 2, 24, 520, 264, "fp16", skew=1.1),
        # gate projections of eight experts, gradients of about 1000 rows each
        _ortho("ortho_wide", 8, 2048, 7168, 1024, "fp32"),
        # the projections of a small layer: latency
        _ortho("ortho_small", 16, 512, 256, 64, "fp32"),
        # odd sizes, tall, bf16 gradients
        _ortho("ortho_odd", 6, 2001, 999, 400, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["gemm", "gemm", "dgrad", "wgrad", "ortho", "ortho"])
        if op == "ortho":
            M, N = _log(rng, 24, 7168), _log(rng, 24, 7168)
            case = _ortho("", _log(rng, 1, 64), M, N, _log(rng, 4, 2048), rng.choice(["fp32", "bf16"]))
            low, most = min(M, N), 4e12
            if low > 2880:
                continue
        else:
            E = rng.choice([1, 3, 8, 16, 32, 64, 96])
            k = rng.choice([j for j in (1, 2, 3, 4, 8) if j <= E])
            case = _grouped("", op, _log(rng, 1, 8192), k, E, 8 * _log(rng, 2, 1792), 8 * _log(rng, 2, 1792),
                            rng.choice(["bf16", "fp16"]),
                            "fp32" if op == "wgrad" else rng.choice(["same", "same", "fp32"]),
                            rng.choice([0.0, 0.5, 1.1]))
            if case["T"] * k > 32768 or E * case["N"] * case["K"] > 1e9:
                continue
            most = 1e12
        del case["name"]
        w = work(case)
        if w["flops"] <= most and w["bytes"] <= 4.5e9:
            return case


def work(case):
    if case["op"] == "ortho":
        low, high = sorted((case["M"], case["N"]))
        # per step: A = X X^T and A A are symmetric (half the products), then (bA + cAA) X
        flops = 5 * (low * low * high + low ** 3 + 2 * low * low * high)
        size = {"fp32": 4, "bf16": 2}[case["dtype"]]
        return {"bytes": case["B"] * case["M"] * case["N"] * (size + 2), "flops": case["B"] * flops}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    M = T * k
    # experts that a token reaches when every expert is equally likely
    active = E * (1 - (1 - k / E) ** T)
    size = 4 if case["out"] == "fp32" else 2
    moved = {"gemm": 2 * M * K + 2 * active * N * K + size * M * N,
             "dgrad": 2 * M * N + 2 * active * N * K + size * M * K,
             "wgrad": 2 * M * (N + K) + 4 * E * N * K}[case["op"]]
    return {"bytes": moved, "flops": 2 * M * N * K}


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    if case["op"] == "ortho":
        B, M, N, rows = case["B"], case["M"], case["N"], case["rows"]
        # a weight gradient: the sum of `rows` outer products dy x^T, whose tokens differ in weight.
        # Of three or more experts the last got no token: its gradient is zero.
        dy = torch.randn(B, rows, M, generator=gen, device=dev)
        dy *= torch.exp(0.5 * torch.randn(B, rows, 1, generator=gen, device=dev)) * 1e-3
        x = torch.randn(B, rows, N, generator=gen, device=dev)
        g = torch.bmm(dy.transpose(1, 2), x)
        if B > 2:
            g[-1] = 0
        return {"case": case, "g": g.to(dt).contiguous()}
    T, k, E, N, K = (case[n] for n in ("T", "k", "E", "N", "K"))
    # routing: every token's k experts are distinct; `skew` makes the first experts more likely
    score = -case["skew"] * torch.log(torch.arange(1, E + 1, device=dev, dtype=torch.float32))
    noise = torch.rand(T, E, generator=gen, device=dev).clamp_(1e-9, 1 - 1e-7)
    idx = torch.topk(score - torch.log(-torch.log(noise)), k, dim=1).indices.reshape(-1)
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    M = T * k
    # for the plain form: the experts that have rows, and each row's place among them
    busy = counts.nonzero().reshape(-1)
    state = {"case": case, "offsets": offsets, "most": int(counts.max()), "busy": busy,
             "seg": torch.repeat_interleave(torch.arange(len(busy), device=dev), counts[busy])}
    state["place"] = torch.arange(M, device=dev) - offsets[busy].long()[state["seg"]]
    if case["op"] != "dgrad":
        state["x"] = torch.randn(M, K, generator=gen, device=dev).to(dt)
    if case["op"] != "gemm":
        state["dy"] = torch.randn(M, N, generator=gen, device=dev).to(dt)
    if case["op"] != "wgrad":
        state["w"] = torch.empty(E, N, K, dtype=dt, device=dev).normal_(0, K ** -0.5, generator=gen)
    return state


# ------------------------------------------------------------------------------ one pass
def run(state):
    return _own(state) if own else _plain(state)


def _pad(rows, state):
    """[M, C] rows -> [experts with rows, longest segment, C] fp32, zero behind each segment."""
    padded = rows.new_zeros((len(state["busy"]), state["most"], rows.shape[1]), dtype=torch.float32)
    padded[state["seg"], state["place"]] = rows.float()
    return padded


def _ns_step(x, _):
    a, b, c = NS
    A = torch.bmm(x, x.transpose(1, 2))
    return a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)


def _plain(state):
    case = state["case"]
    if case["op"] == "ortho":
        g = state["g"].float()
        norm = g.double().square().sum((1, 2), keepdim=True).sqrt()
        x = (g / torch.where(norm > 0, norm, torch.ones_like(norm))).float()
        tall = case["M"] > case["N"]
        x = x.transpose(1, 2) if tall else x
        x = functools.reduce(_ns_step, range(5), x)
        return (x.transpose(1, 2) if tall else x).contiguous().to(torch.bfloat16)
    dt = DTYPES[case["dtype"]]
    at = (state["seg"], state["place"])
    if case["op"] == "gemm":
        y = torch.bmm(_pad(state["x"], state), state["w"][state["busy"]].float().transpose(1, 2))[at]
    elif case["op"] == "dgrad":
        y = torch.bmm(_pad(state["dy"], state), state["w"][state["busy"]].float())[at]
    else:
        dw = state["x"].new_zeros((case["E"], case["N"], case["K"]), dtype=torch.float32)
        dw[state["busy"]] = torch.bmm(_pad(state["dy"], state).transpose(1, 2), _pad(state["x"], state))
        return dw
    return y if case["out"] == "fp32" else y.to(dt)


def _own(state):
    import sparse_mixture_experts_16_b200 as moe

    case = state["case"]
    kept = {"out": state.get("out"), "ws": state.get("ws")}  # a loop keeps its buffers
    out_dtype = torch.float32 if case.get("out") == "fp32" else None
    if case["op"] == "gemm":
        got = moe.moe_grouped_gemm(state["x"], state["offsets"], state["w"], out_dtype=out_dtype, **kept)
    elif case["op"] == "dgrad":
        got = moe.moe_grouped_gemm_dgrad(state["dy"], state["offsets"], state["w"], out_dtype=out_dtype, **kept)
    elif case["op"] == "wgrad":
        got = moe.moe_grouped_gemm_wgrad(state["dy"], state["x"], state["offsets"], **kept)
    else:
        got = moe.moe_orthogonalize(state["g"], steps=5, **kept)
    state["out"], state["ws"] = got
    return state["out"]


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, c = NS
        out = torch.zeros(s["g"].shape, dtype=torch.float64, device=s["g"].device)
        for i in range(case["B"]):
            x = s["g"][i].double()
            size = torch.linalg.vector_norm(x)
            if size == 0:
                continue
            x = x / size
            for _ in range(5):
                # the same iterate with the smaller of X X^T and X^T X: p(X X^T) X = X p(X^T X)
                if case["M"] <= case["N"]:
                    A = x @ x.T
                    x = a * x + b * (A @ x) + c * (A @ (A @ x))
                else:
                    A = x.T @ x
                    x = a * x + b * (x @ A) + c * ((x @ A) @ A)
            out[i] = x
        return out
    edges = s["offsets"].tolist()
    if case["op"] == "wgrad":
        out = torch.empty(case["E"], case["N"], case["K"], dtype=torch.float64, device="cuda")
    else:
        wide = case["N"] if case["op"] == "gemm" else case["K"]
        out = torch.empty(case["T"] * case["k"], wide, dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        at = slice(edges[e], edges[e + 1])
        if case["op"] == "gemm":
            out[at] = s["x"][at].double() @ s["w"][e].double().T
        elif case["op"] == "dgrad":
            out[at] = s["dy"][at].double() @ s["w"][e].double()
        else:
            out[e] = s["dy"][at].double().T @ s["x"][at].double()
    return out
